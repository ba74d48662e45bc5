// norm.hip - the residual's addition with the RMS norm, and the normalised
// vector in fp32 or as the next projection's int8 input.
//
// Per row: t = x + delta; v = t * gamma; per 32 elements the codes of v and
// the sum of t^2 as the activation quantiser makes them (quant.hip), bit for
// bit.  The norm's factor r = 1 / sqrt(sum t^2 / K + eps) is left to the
// consumer (fold), or applied: to the codes' scales, which leaves the codes as
// they are, and to an fp32 output v * r.
//
// Lane l of a wave holds elements 4 l .. 4 l + 3 of 256, so a block of 32 is
// eight lanes.  The quantiser's sums go by pairs of elements 16, 8, 4, 2 and 1
// apart: lanes 4, 2 and 1 apart here, then the elements of a lane.  The row's
// sum of squares is that of its blocks' sums, taken from LDS in an order that
// K alone gives, so that a row's bits do not depend on the other rows.
//
// Bound by memory where the rows are many (8192 rows of 5120, codes: 104 us, 5.4
// TB/s of 13.5 bytes an element, past what a large copy reaches; 3001 of 2560, y:
// 19.5), by the latency of one launch where they are few (in a graph, 5 rows of
// 5120: 2.4 us with the factor left out, 4.3 with it).
#include "sv_internal.h"

namespace sv {

typedef float f4 __attribute__((ext_vector_type(4)));

struct NormArgs {
    const float *x, *delta, *gamma;
    float *sum, *y;
    int8_t *q;
    float *d;
    int32_t *s16;
    float *sumsq;
    int32_t rows, K;
    float eps;
    Div by_quads;  // K / 4
};

__device__ __forceinline__ f4 ld4(const float *p) { return *(const SV_GLOBAL f4 *)p; }
// Vectors are stored past the L2, which holds nothing for the next launch's
// other XCDs anyway (us in a graph: 512 rows of 5120, codes 9.4 -> 7.5; 8192 of
// 2560 49 -> 44, y 65 -> 49; 80 rows the same).
__device__ __forceinline__ void st4(float *p, f4 v) { __builtin_nontemporal_store(v, (SV_GLOBAL f4 *)p); }

// Largest value, and sum, over the eight lanes of a block.
__device__ __forceinline__ float max8(float v) {
    v = fmaxf(v, __shfl_xor(v, 4, 64));
    v = fmaxf(v, __shfl_xor(v, 2, 64));
    return fmaxf(v, __shfl_xor(v, 1, 64));
}
__device__ __forceinline__ f4 sum8(f4 v) {
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1)
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] += __shfl_xor(v[e], o, 64);
    return v;
}

// t = x + delta of a quad.  ONCE: what is read fits no cache, and is loaded past
// them (kCached below).
template <bool ONCE>
__device__ __forceinline__ f4 add_quad(const NormArgs &a, int64_t at) {
    auto ld = [](const float *p) { return ONCE ? __builtin_nontemporal_load((const SV_GLOBAL f4 *)p) : ld4(p); };
    f4 t = ld(a.x + at);
    if (a.delta) t += ld(a.delta + at);
    return t;
}
__device__ __forceinline__ float block_squares(f4 t) {
    const f4 s = sum8(t * t);
    return (s.x + s.z) + (s.y + s.w);
}

// The codes of a quad of v; the scale that is stored is d * r.
__device__ __forceinline__ void store_codes(const NormArgs &a, int64_t at, f4 v, float sq, float r) {
    const float top = max8(fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
    const float d = top / 127.0f, id = d != 0.0f ? 1.0f / d : 0.0f;
    int s = 0;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const int q = static_cast<int>(fminf(fmaxf(roundf(v[e] * id), -127.0f), 127.0f));
        s += q;
        w |= static_cast<uint32_t>(q & 0xFF) << (8 * e);
    }
    s += __shfl_xor(s, 2, 64);
    s += __shfl_xor(s, 1, 64);
    __builtin_nontemporal_store(w, (SV_GLOBAL uint32_t *)(a.q + at));
    const int lane = threadIdx.x & 7;
    if ((lane & 3) == 0) gst(a.s16 + at / 16, s);
    if (lane == 0) {
        gst(a.d + at / 32, d * r);
        gst(a.sumsq + at / 32, sq);
    }
}

// Factor left to the consumer: no row is needed as a whole.
constexpr int kFold = 256;
template <bool ONCE>
__global__ __launch_bounds__(kFold) void add_quant_kernel(NormArgs a) {
    const int i = blockIdx.x * kFold + threadIdx.x, quads = a.K / 4;
    const int row = a.by_quads(i);
    if (row >= a.rows) return;  // eight lanes of a block leave together
    const int64_t at = static_cast<int64_t>(i) * 4;
    const f4 t = add_quad<ONCE>(a, at);
    f4 v = t;
    if (a.gamma) v *= ld4(a.gamma + 4 * (i - row * quads));
    if (a.sum) st4(a.sum + at, t);
    store_codes(a, at, v, block_squares(t), 1.0f);
}

// Factor applied: a workgroup a row, NV quads a thread in registers.
constexpr int kNormBlocks = 1024;  // of a row
template <int THREADS, int NV, bool ONCE>
__global__ __launch_bounds__(THREADS) void add_norm_kernel(NormArgs a) {
    __shared__ float s_sq[kNormBlocks];
    const int tid = threadIdx.x, quads = a.K / 4, nb = a.K / 32;
    for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t base = static_cast<int64_t>(row) * a.K;
        f4 t[NV];
        float sq[NV];
#pragma unroll
        for (int k = 0; k < NV; k++) {
            const int i = tid + k * THREADS;
            t[k] = i < quads ? add_quad<ONCE>(a, base + 4 * i) : f4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        __syncthreads();  // the last row's sums have been read
#pragma unroll
        for (int k = 0; k < NV; k++) {
            const int i = tid + k * THREADS;
            sq[k] = block_squares(t[k]);
            if (i < quads) {
                if ((tid & 7) == 0) s_sq[i / 8] = sq[k];
                if (a.sum) st4(a.sum + base + 4 * i, t[k]);
            }
        }
        __syncthreads();
        float total = 0.0f;
        for (int b = tid & 63; b < nb; b += 64) total += s_sq[b];
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o, 64);
        const float r = 1.0f / sqrtf(total / static_cast<float>(a.K) + a.eps);
#pragma unroll
        for (int k = 0; k < NV; k++) {
            const int i = tid + k * THREADS;
            if (i >= quads) continue;
            const int64_t at = base + 4 * i;
            f4 v = t[k];
            if (a.gamma) v *= ld4(a.gamma + 4 * i);
            if (a.y) st4(a.y + at, v * r);
            if (a.q) store_codes(a, at, v, sq[k], r);
        }
    }
}

constexpr int kNormGrid = 1 << 20;  // threads of a launch fit 32 bits
// 1024 threads a row where few rows leave the chip empty (up to 512 of more than
// 1024 elements) and from the lengths on at which 256 threads would hold six
// quads each: us with 256 and 1024 threads, codes, in a graph: 5 rows of 5120
// 6.1 and 4.3, 256 7.4 and 5.7, 1024 17.2 and 17.2; 8192 rows of 2560 51 and 69,
// of 5120 113 and 114, of 8192 181 and 169; 64 rows of 1024 3.0 and 3.3.
constexpr int kNarrow = 5120;
inline bool wide_rows(int64_t rows, int64_t K) { return K > kNarrow || (rows <= 512 && K > 1024); }

// Bytes of x and delta past which nothing of them is found in the memory-side
// cache of 256 MB, and loads that do not ask it are faster (us in a graph, codes,
// such loads against others: 8192 rows of 5120, 336 MB, 105 and 111; 20000 222
// and 241; 8192 of 2560, 168 MB, 50 and 44).
constexpr int64_t kCached = 1ll << 28;

template <int THREADS, bool ONCE, int NV = 1>
static void launch_norm(const NormArgs &a, hipStream_t st) {
    constexpr int longest = THREADS == 256 ? kNarrow : 32 * kNormBlocks;
    if constexpr (4 * THREADS * NV < longest) {
        if (a.K > 4 * THREADS * NV) return launch_norm<THREADS, ONCE, NV + 1>(a, st);
    }
    hipLaunchKernelGGL((add_norm_kernel<THREADS, NV, ONCE>), dim3(a.rows < kNormGrid ? a.rows : kNormGrid), dim3(THREADS), 0, st, a);
}
template <bool ONCE>
static void launch(const NormArgs &a, bool fold, hipStream_t st) {
    if (fold) {
        const int64_t quads = static_cast<int64_t>(a.rows) * (a.K / 4);
        hipLaunchKernelGGL(add_quant_kernel<ONCE>, dim3(static_cast<unsigned>((quads + kFold - 1) / kFold)), dim3(kFold), 0, st, a);
    } else if (wide_rows(a.rows, a.K)) {
        launch_norm<1024, ONCE>(a, st);
    } else {
        launch_norm<256, ONCE>(a, st);
    }
}

}  // namespace sv

using namespace sv;

extern "C" int sv_add_norm_q8(const float *x, const float *delta, int64_t rows, int64_t K, const float *gamma, float eps,
                              int32_t fold, float *sum, float *y, int8_t *q, float *d, int32_t *s16, float *sumsq,
                              void *stream) {
    SV_REQUIRE(x && (q || y), SV_ERR_ARG, "add_norm_q8: NULL buffer");
    SV_REQUIRE(q ? d && s16 && sumsq : !d && !s16 && !sumsq, SV_ERR_ARG,
               "add_norm_q8: q, d, s16 and sumsq are given together");
    SV_REQUIRE(fold == 0 || fold == 1, SV_ERR_ARG, "add_norm_q8: fold must be 0 or 1");
    SV_REQUIRE(!fold || (q && !y), SV_ERR_ARG, "add_norm_q8: y holds the norm's factor, which fold leaves out");
    SV_REQUIRE(eps >= 0.0f && eps <= 3.0e38f, SV_ERR_ARG, "add_norm_q8: eps must be finite and not negative");
    SV_REQUIRE(K > 0 && K % 32 == 0 && K <= 32 * kNormBlocks, SV_ERR_SHAPE,
               "add_norm_q8: K must be a multiple of 32, at most 32768");
    SV_REQUIRE(rows >= 1 && rows <= (1ll << 33) / K - 1, SV_ERR_SHAPE, "add_norm_q8: rows * K must be below 2^33");
    SV_REQUIRE(aligned(x, 16) && aligned(delta, 16) && aligned(gamma, 16) && aligned(sum, 16) && aligned(y, 16),
               SV_ERR_ALIGN, "add_norm_q8: x, delta, gamma, sum and y must be 16-byte aligned");
    SV_REQUIRE(aligned(q, 4) && aligned(d, 4) && aligned(s16, 4) && aligned(sumsq, 4), SV_ERR_ALIGN,
               "add_norm_q8: q, d, s16 and sumsq must be 4-byte aligned");
    // An output may be x or delta itself (sum only): a thread has read its
    // elements before it writes them.  Other overlaps would race.
    const size_t n = static_cast<size_t>(rows) * static_cast<size_t>(K);
    const void *outs[6] = {sum, y, q, d, s16, sumsq};
    const size_t sizes[6] = {4 * n, 4 * n, n, n / 8, n / 4, n / 8};
    for (int i = 0; i < 6; i++) {
        const bool in_place_x = i == 0 && outs[i] == x, in_place_d = i == 0 && outs[i] == delta;
        SV_REQUIRE((in_place_x || !overlap(outs[i], sizes[i], x, 4 * n)) &&
                       (in_place_d || !overlap(outs[i], sizes[i], delta, 4 * n)) &&
                       !overlap(outs[i], sizes[i], gamma, 4 * static_cast<size_t>(K)),
                   SV_ERR_ARG, "add_norm_q8: an output overlaps an input (sum alone may be x or delta)");
        for (int j = 0; j < i; j++)
            SV_REQUIRE(!overlap(outs[i], sizes[i], outs[j], sizes[j]), SV_ERR_ARG, "add_norm_q8: outputs overlap");
    }
    NormArgs a{x, delta, gamma, sum, y, q, d, s16, sumsq, static_cast<int32_t>(rows), static_cast<int32_t>(K), eps,
               div_by(static_cast<uint32_t>(K / 4))};
    hipStream_t st = as_stream(stream);
    if (rows * K * (delta ? 8 : 4) > kCached) launch<true>(a, fold, st);
    else launch<false>(a, fold, st);
    return hip_check(hipGetLastError(), "add_norm_q8 launch");
}
