// sample.hip - sampling with temperature, top-k, top-p and min-p from given
// uniforms.
//
// A row's weights are w_j = exp((z_j - max z) / T), 1 for the largest.  The
// filters keep, in the order of falling z (equal ones by rising index), the
// first top_k; of these the shortest run whose weights reach top_p of their
// sum; of these the weights of at least min_p.  So what the first two keep is
// given by a border: all z above it, and of those equal to it the first few
// indices.  The token is the least index at which the running sum of the kept
// weights, in the order of the indices, exceeds u times their sum.
//
// Sums are whole numbers: each weight, formed in fp64, counts as the nearest
// multiple of 2^-s with s = 63 - ceil(log2 V), at most 51 (2^-45 for 151936
// tokens), so a sum of V of them fits 64 bits and is the same in any order:
// atomics and any split of a row give the same bits.  A weight below half a step is never
// drawn: all of them together are less than V^2 2^-64 of the row (1e-9 for
// 151936).
//
// The borders are found by radix selection on the bits of z (11, 11 and 10 of
// them), by numbers of elements for top-k and by sums of weights for top-p.
#include <algorithm>

#include "sv_internal.h"

namespace sv {

constexpr int kSample = 1024;  // threads of a row's workgroup
constexpr int kWaves = kSample / 64;
constexpr int kDigits = 2048;
constexpr int64_t kMaxVocab = 1 << 24;
constexpr int64_t kMaxRows = 65535;

struct SampleArgs {
    const float *logits;
    int64_t ld;
    const sv_sampling *params;
    int32_t per_row;  // 0: one for all rows
    int32_t V;
    int32_t shift;    // weights in steps of 2^-shift
    const double *u;
    int32_t *tokens;
    float *probs, *kept;
};

typedef unsigned long long u64;

// A row's kept set: keys above `key`, and those equal to it with an index
// below `cut`.
struct Border {
    uint32_t key;
    int32_t cut;
    __device__ bool keeps(uint32_t k, int j) const { return k > key || (k == key && j < cut); }
};

__device__ __forceinline__ double weight_of(float z, float zmax, double per) {
    return exp2((static_cast<double>(z) - static_cast<double>(zmax)) * per);
}
// w in [0, 1] to the nearest multiple of 2^-shift: 2^(52 - shift) + w leaves
// the multiple in the low bits of its fraction.
__device__ __forceinline__ u64 steps_of(double w, int shift) {
    const double one = __longlong_as_double(static_cast<long long>(1023 + 52 - shift) << 52);
    return static_cast<u64>(__double_as_longlong(one + w)) & ((1ull << 52) - 1);
}

struct SampleShared {
    u64 hist[kDigits];
    u64 wave[kWaves];
    u64 total, above;
    int32_t digit, at;
    float top;
    int32_t finite, bad;
};

__device__ __forceinline__ u64 wave_sum(u64 v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ u64 wave_scan(u64 v) {  // sum of the lanes up to and with this one
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const u64 t = __shfl_up(v, o, 64);
        if (lane >= o) v += t;
    }
    return v;
}
// Sum over the workgroup's threads before this one; *all is that over all.
__device__ __forceinline__ u64 block_scan(SampleShared &sh, u64 v, u64 *all) {
    const int wave = threadIdx.x >> 6;
    const u64 upto = wave_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) sh.wave[wave] = upto;
    __syncthreads();
    u64 before = 0, sum = 0;
    for (int w = 0; w < kWaves; w++) {
        if (w < wave) before += sh.wave[w];
        sum += sh.wave[w];
    }
    *all = sum;
    return before + upto - v;
}

// Moves the border so that the first `want` (of falling order) of what it
// keeps remain: of `want` elements, or of steps of weight.
template <bool MASS>
__device__ void select(const SampleArgs &a, SampleShared &sh, const float *row, float zmax, double per, u64 want,
                       Border *border) {
    const int tid = threadIdx.x;
    const Border from = *border;
    uint32_t prefix = 0, known = 0;  // the bits of the key found so far, and which they are
    u64 above = 0;                   // amount above them
    for (int level = 0; level < 3; level++) {
        const int low = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        for (int i = tid; i < kDigits; i += kSample) sh.hist[i] = 0;
        __syncthreads();
        for (int j = tid; j < a.V; j += kSample) {
            const float z = gld(row + j);
            const uint32_t k = float_key(z);
            if ((k & known) != prefix || !from.keeps(k, j)) continue;
            const u64 n = MASS ? steps_of(weight_of(z, zmax, per), a.shift) : 1;
            atomicAdd(&sh.hist[(k >> low) & ((1u << bits) - 1)], n);
        }
        __syncthreads();
        // digits in falling order, two a thread
        const int d1 = kDigits - 1 - 2 * tid, d0 = d1 - 1;
        const u64 h1 = sh.hist[d1], h0 = sh.hist[d0];
        u64 all;
        const u64 before = above + block_scan(sh, h1 + h0, &all);
        if (before < want && before + h1 >= want) {
            sh.digit = d1;
            sh.above = before;
        } else if (before + h1 < want && before + h1 + h0 >= want) {
            sh.digit = d0;
            sh.above = before + h1;
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(sh.digit) << low;
        known |= ((1u << bits) - 1) << low;
        above = sh.above;
        __syncthreads();
    }
    // of the elements equal to the border the first `need`
    const u64 ties_amount = MASS ? steps_of(weight_of(__uint_as_float(prefix & 0x80000000u ? prefix ^ 0x80000000u : ~prefix),
                                                      zmax, per), a.shift) : 1;
    const u64 need = (want - above + ties_amount - 1) / ties_amount;
    u64 passed = 0;
    int cut = a.V;
    for (int j0 = 0; j0 < a.V; j0 += kSample) {
        const int j = j0 + tid;
        bool is = false;
        if (j < a.V) {
            const uint32_t k = float_key(gld(row + j));
            is = k == prefix && from.keeps(k, j);
        }
        u64 all;
        const u64 before = passed + block_scan(sh, is ? 1 : 0, &all);
        if (is && before + 1 == need) sh.at = j + 1;
        passed += all;
        __syncthreads();
        if (passed >= need) {
            cut = sh.at;
            break;
        }
    }
    __syncthreads();
    *border = Border{prefix, cut};
}

__global__ __launch_bounds__(kSample) void sample_kernel(SampleArgs a) {
    __shared__ SampleShared sh;
    const int tid = threadIdx.x, r = blockIdx.x, V = a.V;
    const float *row = a.logits + static_cast<int64_t>(r) * a.ld;
    const sv_sampling p = a.params[a.per_row ? r : 0];
    bool fine = p.temperature >= 0.0f && p.temperature < INFINITY && p.top_k >= 0 && p.top_p > 0.0f && p.top_p <= 1.0f &&
                p.min_p >= 0.0f && p.min_p <= 1.0f;

    // ---- largest value, and what cannot be sampled from
    float top = -INFINITY;
    int finite = 0, bad = 0;
    for (int j = tid; j < V; j += kSample) {
        const float z = gld(row + j);
        if (!(z < INFINITY)) bad = 1;
        if (z > -INFINITY) finite++;
        top = fmaxf(top, z);
    }
    if (tid == 0) {
        sh.finite = sh.bad = 0;
        sh.top = -INFINITY;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if ((tid & 63) == 0) sh.wave[tid >> 6] = __float_as_uint(top);
    __syncthreads();
    atomicAdd(&sh.finite, finite);
    if (bad) atomicOr(&sh.bad, 1);
    __syncthreads();
    for (int w = 0; w < kWaves; w++) top = fmaxf(top, __uint_as_float(static_cast<uint32_t>(sh.wave[w])));
    finite = sh.finite;
    fine = fine && !sh.bad && finite > 0;
    const float zmax = top + 0.0f;
    const bool greedy = p.temperature == 0.0f;
    const double per = greedy ? 1.0 : 1.44269504088896340736 / static_cast<double>(p.temperature);

    Border border{float_key(-INFINITY), 0};
    u64 total = 0;
    int token = -1;
    if (fine) {
        const int k = greedy ? 1 : p.top_k == 0 ? V : p.top_k;
        __syncthreads();
        if (k < finite) select<false>(a, sh, row, zmax, per, static_cast<u64>(k), &border);
        auto sum_kept = [&](double least) {
            u64 n = 0, all;
            for (int j = tid; j < V; j += kSample) {
                const float z = gld(row + j);
                if (!border.keeps(float_key(z), j)) continue;
                const double w = weight_of(z, zmax, per);
                if (w >= least) n += steps_of(w, a.shift);
            }
            block_scan(sh, n, &all);
            return all;
        };
        if (p.top_p < 1.0f) {
            const u64 all = sum_kept(0.0);
            const double goal = ceil(static_cast<double>(p.top_p) * static_cast<double>(all));
            u64 want = goal < 1.0 ? 1 : static_cast<u64>(goal);
            if (want > all) want = all;
            select<true>(a, sh, row, zmax, per, want, &border);
        }
        const double least = static_cast<double>(p.min_p);
        total = sum_kept(least);
        const double u = a.tokens ? a.u[r] : -1.0;
        if (u >= 0.0 && u < 1.0) {
            u64 before_thr = static_cast<u64>(u * static_cast<double>(total));
            if (before_thr >= total) before_thr = total - 1;
            u64 passed = 0;
            for (int j0 = 0; j0 < V; j0 += kSample) {
                const int j = j0 + tid;
                u64 n = 0, all;
                if (j < V) {
                    const float z = gld(row + j);
                    const double w = weight_of(z, zmax, per);
                    if (border.keeps(float_key(z), j) && w >= least) n = steps_of(w, a.shift);
                }
                const u64 before = passed + block_scan(sh, n, &all);
                if (before <= before_thr && before + n > before_thr) sh.at = j;
                passed += all;
                __syncthreads();
                if (passed > before_thr) {
                    token = sh.at;
                    break;
                }
            }
        }
    }
    if (tid == 0 && a.tokens) a.tokens[r] = token;
    if (!a.probs && !a.kept) return;
    const double least = static_cast<double>(p.min_p);
    const double scale = ldexp(1.0, a.shift) / static_cast<double>(total);
    for (int j = tid; j < V; j += kSample) {
        const float z = gld(row + j);
        const double w = weight_of(z, zmax, per);
        const bool keep = border.keeps(float_key(z), j) && w >= least;
        const int64_t at = static_cast<int64_t>(r) * V + j;
        if (a.probs) gst(a.probs + at, fine ? (keep ? static_cast<float>(w * scale) : 0.0f) : NAN);
        if (a.kept) gst(a.kept + at, fine ? (keep ? z : -INFINITY) : NAN);
    }
}

static int check_rows(int64_t rows, int64_t V) {
    SV_REQUIRE(rows >= 1 && rows <= kMaxRows, SV_ERR_SHAPE, "sample: rows must be in [1, 65535]");
    SV_REQUIRE(V >= 1 && V <= kMaxVocab, SV_ERR_SHAPE, "sample: V must be in [1, 2^24]");
    return SV_OK;
}

}  // namespace sv

using namespace sv;

extern "C" size_t sv_sample_workspace_bytes(int64_t rows, int64_t V) {
    if (check_rows(rows, V)) return 0;
    return 256;
}

extern "C" int sv_sample(const float *logits, int64_t rows, int64_t V, int64_t ld, const sv_sampling *params,
                         int32_t n_params, const double *u, int32_t *tokens, float *probs, float *kept, void *workspace,
                         size_t ws_bytes, void *stream) {
    const int rc = check_rows(rows, V);
    if (rc) return rc;
    SV_REQUIRE(logits && params && workspace && (tokens || probs || kept) && (!tokens || u), SV_ERR_ARG,
               "sample: NULL buffer");
    SV_REQUIRE(ld >= V && ld < (1ll << 31), SV_ERR_SHAPE, "sample: ld must be in [V, 2^31)");
    SV_REQUIRE(n_params == 1 || n_params == rows, SV_ERR_ARG, "sample: n_params must be 1 or rows");
    SV_REQUIRE(aligned(logits, 4) && aligned(params, 4) && aligned(u, 8) && aligned(tokens, 4) && aligned(probs, 4) &&
                   aligned(kept, 4) && aligned(workspace, 256),
               SV_ERR_ALIGN, "sample: alignment (4 bytes, u 8, workspace 256)");
    const size_t need = sv_sample_workspace_bytes(rows, V);
    SV_REQUIRE(ws_bytes >= need, SV_ERR_WORKSPACE, "sample: workspace needs " + std::to_string(need) + " bytes");
    const size_t in = (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) + static_cast<size_t>(V)) * 4;
    const size_t out = static_cast<size_t>(rows) * static_cast<size_t>(V) * 4;
    SV_REQUIRE(!overlap(logits, in, probs, out) && !overlap(logits, in, kept, out) && !overlap(probs, out, kept, out), SV_ERR_ARG,
               "sample: probs, kept and logits overlap");
    int bits = 0;
    while ((1ll << bits) < V) bits++;
    SampleArgs a{logits, ld, params, n_params > 1, static_cast<int32_t>(V), std::min(51, 63 - bits), u, tokens,
                 probs, kept};
    hipLaunchKernelGGL(sample_kernel, dim3(static_cast<unsigned>(rows)), dim3(kSample), 0, as_stream(stream), a);
    return hip_check(hipGetLastError(), "sample launch");
}
