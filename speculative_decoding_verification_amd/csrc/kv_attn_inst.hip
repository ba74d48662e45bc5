// kv_attn_inst.hip - attention of the new rows over the cache, one chunk of
// the length per workgroup; compiled once per cache type (SV_INST_KV).
//
// For a row with query q and the visible slots j of a chunk:
//   s_j = q . k_j,  m = max s_j,  l = sum 2^(s_j - m),  o = sum 2^(s_j - m) v_j
// in one pass over the chunk with a running m, l and o (q is scaled by
// scale * log2(e) first).  The rows of one key head, M * group of them, are
// the 16 columns of a tile; a wave takes every fourth block of 32 slots:
//   S^T [32 slots x 16 rows] = K Q^T    two 16x16x32 products per 32 of dim
//   O^T [dim x 16 rows] += V^T P^T      one 16x16x32 product per 16 of dim
// Row r of the first product's tile t is slot 8 (r / 4) + 4 t + r % 4, so
// lane group g (lanes 16 g ..) holds the scores of slots 8 g .. 8 g + 7, and
// these are the eight it supplies to the second product: the weights stay
// where they are, and keys and values go from the block straight to
// registers, 16 (int8: 8) contiguous bytes a lane.
//
// Precision: the fp32 q and weights enter as sums of parts, two for fp16 (q
// scaled by a power of two per row, the weights by 2^15, so that the second
// part stays a normal number) and three for bf16; int8 codes are exact in
// either, keys go with fp16 and values, whose weights carry the value's
// scale and so have no bounded range, with bf16.
//
// Bound by memory: a block of 32 slots is 128 dim bytes (64 dim for int8)
// and is read once; at 16 rows the products take a tenth of that time.
#include "kv_attn.h"

namespace sv {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

template <int TYPE>
struct Kind;
template <>
struct Kind<SV_KV_F16> {
    typedef h8 KVec;
    typedef h8 VVec;
    static constexpr int kq = 2, kp = 2, esz = 2;
};
template <>
struct Kind<SV_KV_BF16> {
    typedef b8 KVec;
    typedef b8 VVec;
    static constexpr int kq = 3, kp = 3, esz = 2;
};
template <>
struct Kind<SV_KV_I8> {
    typedef h8 KVec;
    typedef b8 VVec;
    static constexpr int kq = 2, kp = 3, esz = 1;
};

__device__ __forceinline__ f4 mma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f4 mma(b8 a, b8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

constexpr int kWaves = 4;

// x = sum of N parts of the narrow type, each the rounding of what is left.
template <int N, typename V8>
__device__ __forceinline__ void split8(const float (&x)[8], V8 (&part)[N]) {
    float left[8];
#pragma unroll
    for (int e = 0; e < 8; e++) left[e] = x[e];
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const auto h = static_cast<decltype(part[0][0] + part[0][0])>(left[e]);
            part[n][e] = h;
            left[e] -= static_cast<float>(h);
        }
}

// w y as the products of w's parts make it, for a y that is not finite.
template <int N, typename V8>
__device__ __forceinline__ float times_parts(float w, float y) {
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < N; n++) {
        V8 h;
        h[0] = static_cast<decltype(h[0] + h[0])>(w);
        w -= static_cast<float>(h[0]);
        sum += static_cast<float>(h[0]) * y;
    }
    return sum;
}

// Raw piece of a block as one lane loads it.
template <int ESZ>
struct Raw {
    uint32_t w[2 * ESZ];
};
template <int ESZ>
__device__ __forceinline__ Raw<ESZ> load_raw(const uint8_t *p) {
    Raw<ESZ> r;
    if constexpr (ESZ == 2) {
        const u32x4 v = *(const SV_GLOBAL u32x4 *)p;
        r.w[0] = v.x;
        r.w[1] = v.y;
        r.w[2] = v.z;
        r.w[3] = v.w;
    } else {
        const u32x2 v = *(const SV_GLOBAL u32x2 *)p;
        r.w[0] = v.x;
        r.w[1] = v.y;
    }
    return r;
}

template <typename V8>
__device__ __forceinline__ V8 widen(const Raw<2> &r) {
    V8 v;
    __builtin_memcpy(&v, r.w, 16);
    return v;
}
// Four codes to fp16: 0x6400 | (c + 128) is 1024 + 128 + c.
template <typename V8>
__device__ __forceinline__ V8 widen(const Raw<1> &r) {
    V8 v;
    if constexpr (__is_same(V8, h8)) {
        const h2 bias = {static_cast<_Float16>(1152.0f), static_cast<_Float16>(1152.0f)};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t u = r.w[i >> 1] ^ 0x80808080u;
            const uint32_t w = __builtin_amdgcn_perm(0x64646464u, u, (i & 1) ? 0x04030402u : 0x04010400u);
            h2 x;
            __builtin_memcpy(&x, &w, 4);
            x = x - bias;
            v[2 * i] = x[0];
            v[2 * i + 1] = x[1];
        }
    } else {
        uint32_t z[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int32_t u = static_cast<int32_t>(r.w[i >> 1]);
            const float lo = static_cast<float>(static_cast<int8_t>(u >> ((i & 1) * 16)));
            const float hi = static_cast<float>(static_cast<int8_t>(u >> ((i & 1) * 16 + 8)));
            z[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
        }
        __builtin_memcpy(&v, z, 16);
    }
    return v;
}

// An element pair's bits that make it an infinity or NaN.
template <int TYPE>
__device__ __forceinline__ uint32_t odd_pair(uint32_t w) {
    return ((w & 0x7FFF7FFFu) + (TYPE == SV_KV_F16 ? 0x04000400u : 0x00800080u)) & 0x80008000u;
}

// Largest value over the four lanes that share a row (16 and 32 lanes apart).
__device__ __forceinline__ float row_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

template <int TYPE, int D, int RT>
struct Lds {
    // queries as operands, [tile][dim / 32][part][lane][16 bytes], and behind
    // them the fp32 rows they are made of; after the blocks the waves' sums,
    // two waves at a time
    static constexpr int q_bytes = RT * (D / 32) * Kind<TYPE>::kq * 1024;
    static constexpr int ld = D + 4;
    static constexpr int row_bytes = 16 * RT * ld * 4;
    static constexpr int bytes = q_bytes > row_bytes ? q_bytes + row_bytes : 2 * row_bytes;
};

// The rows' queries, rotated and scaled, as fp32 in LDS: the workgroup's
// threads take four elements each, and every load of an element is issued
// before any is used.
template <int D, int ROWS, int MODE>
__device__ __forceinline__ void stage_rows(const AttnArgs &a, const Span &sp, int b, int head, int row0, int rows,
                                           const int *depth, float *to) {
    constexpr int LD = D + 4, QUADS = D / 4;
#pragma unroll 4
    for (int it = threadIdx.x; it < ROWS * QUADS; it += 64 * kWaves) {
        const int i = it / QUADS, d = it % QUADS * 4;
        const int r = row0 + i;
        const bool live = r < rows;
        const int m = live ? r / a.group : 0;
        const int hq = head * a.group + (live ? r % a.group : 0);
        const float *qp = a.q + ((static_cast<int64_t>(b) * a.bt.M + m) * a.q_heads + hq) * D;
        const uint4 u = gld16(qp + d);
        float x[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
        if constexpr (MODE != SV_ROPE_NONE) {
            const int half = a.rope.rot / 2;
            const int64_t pos = min(sp.len + depth[m], static_cast<int64_t>(a.rope.n_pos - 1));
            const float *cs = a.rope.table + pos * half * 2;
            if constexpr (MODE == SV_ROPE_PAIRS) {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const bool turn = d + e < a.rope.rot;
                    const uint2 w = gld8(cs + (turn ? d + e : 0));
                    const float co = __uint_as_float(w.x), si = __uint_as_float(w.y), x0 = x[e], x1 = x[e + 1];
                    if (turn) {
                        x[e] = __fsub_rn(__fmul_rn(x0, co), __fmul_rn(x1, si));
                        x[e + 1] = __fadd_rn(__fmul_rn(x1, co), __fmul_rn(x0, si));
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const bool turn = d + e < a.rope.rot, second = d + e >= half;
                    const int p = !turn ? 0 : second ? d + e - half : d + e;
                    const uint2 w = gld8(cs + 2 * p);
                    const float other = gld(qp + (!turn ? 0 : second ? p : p + half));
                    const float own = __fmul_rn(x[e], __uint_as_float(w.x));
                    const float by = __fmul_rn(other, __uint_as_float(w.y));
                    if (turn) x[e] = second ? __fadd_rn(own, by) : __fsub_rn(own, by);
                }
            }
        }
        typedef float f4 __attribute__((ext_vector_type(4)));
        f4 z;
#pragma unroll
        for (int e = 0; e < 4; e++) z[e] = live ? x[e] * a.scale : 0.0f;
        *reinterpret_cast<f4 *>(to + i * LD + d) = z;
    }
}

// The queries of a row tile as the second operand of S^T = K Q^T (one wave),
// for fp16 multiplied by the power of two that brings the row's largest
// magnitude into [2^12, 2^13); rs is what the row's scores are multiplied by
// to undo that.
template <int TYPE, int D>
__device__ __forceinline__ void put_queries(const float *from, uint8_t *to, float *rs) {
    using Kd = Kind<TYPE>;
    constexpr int NC = D / 32, LD = D + 4;
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    float xq[NC][8];
    float top = 0.0f;
#pragma unroll
    for (int cc = 0; cc < NC; cc++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
            xq[cc][e] = from[col * LD + 32 * cc + 8 * g + e];
            top = fmaxf(top, fabsf(xq[cc][e]));
        }
    float back = 1.0f;
    if constexpr (__is_same(typename Kd::KVec, h8)) {
        top = row_max(top);
        const int ex = static_cast<int>(__float_as_uint(top) >> 23);  // biased; 255 = not finite
        const int up = ex == 0 || ex == 255 ? 0 : max(-100, min(100, 12 - (ex - 127)));
        const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
        for (int cc = 0; cc < NC; cc++)
#pragma unroll
            for (int e = 0; e < 8; e++) xq[cc][e] *= by;
    }
    if (g == 0) rs[col] = back;
#pragma unroll
    for (int cc = 0; cc < NC; cc++) {
        typename Kd::KVec part[Kd::kq];
        split8<Kd::kq>(xq[cc], part);
#pragma unroll
        for (int n = 0; n < Kd::kq; n++)
            *reinterpret_cast<typename Kd::KVec *>(to + ((cc * Kd::kq + n) * 64 + lane) * 16) = part[n];
    }
}

// Two waves a SIMD cover each other's waits where the registers allow it.
template <int TYPE, int D, int RT>
constexpr int min_waves() {
    return RT * D <= 256 && (TYPE == SV_KV_I8 || D <= 192) ? 2 : 1;
}

template <int TYPE, int D, int RT>
__global__ __launch_bounds__(64 * kWaves, (min_waves<TYPE, D, RT>())) void kv_attn_kernel(AttnArgs a) {
    using Kd = Kind<TYPE>;
    using L = Lds<TYPE, D, RT>;
    constexpr int NC = D / 32, ND = D / 16, ESZ = Kd::esz;
    constexpr int LD = L::ld;
    constexpr int ROWS = 16 * RT;
    __shared__ __align__(16) uint8_t s_mem[L::bytes];
    __shared__ float s_m[kWaves][ROWS], s_l[kWaves][ROWS], s_rs[ROWS];
    __shared__ uint32_t s_mask[SV_MAX_M];  // the new rows that a row sees, and how many come before it
    __shared__ int s_depth[SV_MAX_M];
    float *s_o = reinterpret_cast<float *>(s_mem);  // [2][ROWS][LD]

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    // Row groups of one (sequence, head, chunk) read the same blocks: eight
    // workgroups apart, so that the same XCD takes them and its L2 serves
    // the second reading.
    const int x = blockIdx.x;
    const int tile = x / 8 % a.tiles, unit = x / 8 / a.tiles * 8 + x % 8;
    const int heads = a.kv.heads;
    const int c = unit % a.chunks, bh = unit / a.chunks;
    const int head = bh % heads, b = bh / heads;
    if (b >= a.bt.B) return;
    const int sid = a.bt.seq ? __builtin_amdgcn_readfirstlane(gld(a.bt.seq + b)) : b;
    if (sid < 0 || sid >= a.kv.seqs) return;
    const Span sp = span_of(a, b, sid);
    const int ac = chunk_of(sp, c);
    const bool alone = a.chunks == 1;  // no join: this workgroup finishes the rows
    if (ac >= sp.end && !alone) return;
    const int row0 = tile * ROWS;
    const int rows = sp.n * a.group;  // of this sequence, in use
    if (row0 >= rows) return;

    // ---- the wave's blocks: every fourth one of the chunk, but for those
    // between the sinks and every row's window
    const int per = a.chunk / kBlk;
    const int last = static_cast<int>(min(static_cast<int64_t>(ac + 1) * per, (sp.total + kBlk - 1) / kBlk));
    const int gap0 = (a.sinks + kBlk - 1) / kBlk, gap1 = static_cast<int>(sp.lo / kBlk);
    const int begin = ac * per + wave;
    auto settle = [&](int j) {  // j, or the next of the wave's blocks past the gap
        return j >= gap0 && j < gap1 ? j + (gap1 - j + kWaves - 1) / kWaves * kWaves : j;
    };
    auto page_of = [&](int j) {
        return j < last ? __builtin_amdgcn_readfirstlane(kv_page_of(a.kv, sid, j >> a.kv.blk_shift)) : -1;
    };
    // a block without a page is read from page 0 and masked
    auto block_at = [&](int j, int page) {
        return kv_block(a.kv, a.layer, max(page, 0), head, j & ((1 << a.kv.blk_shift) - 1));
    };
    Raw<ESZ> kr[NC][2], vr[ND];
    float ks[8], vs[8];  // int8: the scales of the lane group's eight slots
    const uint32_t k_at = (g * 32 + 8 * (col >> 2) + (col & 3)) * 8 * ESZ;
    const uint32_t v_at = (32 * D + (g * D + col) * 8) * ESZ;
    auto load_k = [&](const uint8_t *blk) {
#pragma unroll
        for (int cc = 0; cc < NC; cc++)
#pragma unroll
            for (int u = 0; u < 2; u++) kr[cc][u] = load_raw<ESZ>(blk + k_at + (cc * 128 + 4 * u) * 8 * ESZ);
        if constexpr (TYPE == SV_KV_I8) {
            const uint8_t *sc = blk + 64 * D + 32 * g;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const uint4 w = gld16(sc + 4 * e);
                ks[e] = __uint_as_float(w.x);
                ks[e + 1] = __uint_as_float(w.y);
                ks[e + 2] = __uint_as_float(w.z);
                ks[e + 3] = __uint_as_float(w.w);
            }
        }
    };
    auto load_v = [&](const uint8_t *blk) {
        if constexpr (TYPE == SV_KV_I8) {
            const uint8_t *sc = blk + 64 * D + 128 + 32 * g;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const uint4 w = gld16(sc + 4 * e);
                vs[e] = __uint_as_float(w.x);
                vs[e + 1] = __uint_as_float(w.y);
                vs[e + 2] = __uint_as_float(w.z);
                vs[e + 3] = __uint_as_float(w.w);
            }
        }
#pragma unroll
        for (int i = 0; i < ND; i++) vr[i] = load_raw<ESZ>(blk + v_at + i * 128 * ESZ);
    };

    int j = settle(begin);
    int page = page_of(j);
    const uint8_t *blk = block_at(j, page);
    int jn = settle(j + kWaves);
    int page_n = page_of(jn);
    if (j < last) {
        load_k(blk);
        load_v(blk);
    }
    if (threadIdx.x < SV_MAX_M) {
        const uint32_t mask = static_cast<int>(threadIdx.x) < sp.n ? row_mask(a, b, threadIdx.x) : 0u;
        s_mask[threadIdx.x] = mask;
        s_depth[threadIdx.x] = __popc(mask & ((1u << threadIdx.x) - 1));
    }
    __syncthreads();
    float *staged = reinterpret_cast<float *>(s_mem + L::q_bytes);
    if (a.rope.mode == SV_ROPE_NONE) stage_rows<D, ROWS, SV_ROPE_NONE>(a, sp, b, head, row0, rows, s_depth, staged);
    else if (a.rope.mode == SV_ROPE_PAIRS) stage_rows<D, ROWS, SV_ROPE_PAIRS>(a, sp, b, head, row0, rows, s_depth, staged);
    else stage_rows<D, ROWS, SV_ROPE_HALVES>(a, sp, b, head, row0, rows, s_depth, staged);
    __syncthreads();
    if (wave < RT) put_queries<TYPE, D>(staged + 16 * wave * LD, s_mem + wave * (L::q_bytes / RT), s_rs + 16 * wave);
    __syncthreads();

    f4 o[RT][ND];
    float mx[RT], l[RT], rs[RT];
#pragma unroll
    for (int t = 0; t < RT; t++) {
        mx[t] = -INFINITY;
        l[t] = 0.0f;
        rs[t] = s_rs[16 * t + col];
#pragma unroll
        for (int i = 0; i < ND; i++) o[t][i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int64_t whole = sp.len + sp.n - a.window;  // with a window: from here on every row's window has begun
    while (j < last) {
        const int64_t s0 = static_cast<int64_t>(j) * kBlk;
        // ---- scores, and the next block's keys on their way
        float p[RT][8];
        {
            f4 acc[RT][2];
#pragma unroll
            for (int t = 0; t < RT; t++) acc[t][0] = acc[t][1] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int cc = 0; cc < NC; cc++) {
                const typename Kd::KVec k0 = widen<typename Kd::KVec>(kr[cc][0]);
                const typename Kd::KVec k1 = widen<typename Kd::KVec>(kr[cc][1]);
#pragma unroll
                for (int n = Kd::kq - 1; n >= 0; n--)
#pragma unroll
                    for (int t = 0; t < RT; t++) {
                        const typename Kd::KVec q = *reinterpret_cast<const typename Kd::KVec *>(
                            s_mem + t * (L::q_bytes / RT) + ((cc * Kd::kq + n) * 64 + lane) * 16);
                        acc[t][0] = mma(k0, q, acc[t][0]);
                        acc[t][1] = mma(k1, q, acc[t][1]);
                    }
            }
#pragma unroll
            for (int t = 0; t < RT; t++)
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    p[t][e] = acc[t][e >> 2][e & 3] * rs[t];
                    if constexpr (TYPE == SV_KV_I8) p[t][e] *= ks[e];
                }
        }
        const uint8_t *blk_n = block_at(jn, page_n);
        __builtin_amdgcn_sched_barrier(0);
        if (jn < last) load_k(blk_n);
        const int jnn = settle(jn + kWaves);
        const int page_nn = page_of(jnn);
        __builtin_amdgcn_sched_barrier(0);

        // ---- what is visible, and the running softmax
        const bool edge = page < 0 || s0 + kBlk > sp.len || (a.window && s0 < whole && s0 + kBlk > a.sinks);
        // slots of the lane group that any row of the tile sees, and those that all see
        uint32_t any_sees = edge ? 0u : 0xFFu, all_see = 0xFFu;
        uint32_t seen[RT];  // slots of the lane group that the lane's row sees
#pragma unroll
        for (int t = 0; t < RT; t++) seen[t] = 0xFFu;
        if (edge) {
#pragma unroll
            for (int t = 0; t < RT; t++) {
                const int r = row0 + 16 * t + col;
                const bool live = r < rows;
                const int m = live ? r / a.group : 0;
                const uint32_t mask = s_mask[m];
                const int64_t pos = sp.len + s_depth[m];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int64_t slot = s0 + 8 * g + e;
                    const int nth = static_cast<int>(slot - sp.len);
                    bool sees = page >= 0 && slot < sp.total && (nth < 0 || (nth < sp.n && (mask >> nth & 1u)));
                    if (a.window && sees) {
                        const int64_t kpos = nth < 0 ? slot : sp.len + s_depth[nth];
                        sees = pos - kpos < a.window || kpos < a.sinks;
                    }
                    if (!sees) {
                        p[t][e] = -INFINITY;
                        seen[t] &= ~(1u << e);
                    }
                    const uint32_t by = static_cast<uint32_t>(__ballot(live && sees) >> (16 * g)) & 0xFFFFu;
                    const uint32_t of = static_cast<uint32_t>(__ballot(live) >> (16 * g)) & 0xFFFFu;
                    if (by) any_sees |= 1u << e;
                    if (by != of) all_see &= ~(1u << e);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < RT; t++) {
            float top = p[t][0];
#pragma unroll
            for (int e = 1; e < 8; e++) top = fmaxf(top, p[t][e]);
            const float now = fmaxf(mx[t], row_max(top));
            const float base = now == -INFINITY ? 0.0f : now;
            const float keep = __builtin_amdgcn_exp2f(mx[t] - base);
            mx[t] = now;
            // fp16 weights are taken times 2^15 (l too, so it cancels)
            constexpr float kUp = TYPE == SV_KV_F16 ? 15.0f : 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                p[t][e] = __builtin_amdgcn_exp2f(p[t][e] - base + kUp);
                sum += p[t][e];
            }
            l[t] = l[t] * keep + sum;
            if (__any(keep != 1.0f)) {
#pragma unroll
                for (int i = 0; i < ND; i++) o[t][i] *= keep;
            }
            if constexpr (TYPE == SV_KV_I8) {
#pragma unroll
                for (int e = 0; e < 8; e++) p[t][e] = p[t][e] == 0.0f ? 0.0f : p[t][e] * vs[e];
            }
        }

        // ---- o += V^T P^T
        bool odd = false;
        if constexpr (TYPE != SV_KV_I8) {
            if (edge) {
                // Values in slots that no row sees count as 0, whatever they
                // hold.  Infinities and NaN in a slot that some rows see and
                // others do not cannot go through a product with weight 0:
                // they are taken out and added row by row.
                uint32_t keep2[4], some[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    keep2[e] = (any_sees >> (2 * e) & 1u ? 0x0000FFFFu : 0u) | (any_sees >> (2 * e + 1) & 1u ? 0xFFFF0000u : 0u);
                    some[e] = (all_see >> (2 * e) & 1u ? 0u : 0x00008000u) | (all_see >> (2 * e + 1) & 1u ? 0u : 0x80000000u);
                }
                uint32_t found = 0;
#pragma unroll
                for (int i = 0; i < ND; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        vr[i].w[e] &= keep2[e];
                        found |= odd_pair<TYPE>(vr[i].w[e]) & some[e];
                    }
                odd = __any(found != 0);
                if (odd) {
#pragma unroll
                    for (int i = 0; i < ND; i++)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const uint32_t f = odd_pair<TYPE>(vr[i].w[e]);
                            if (f & 0x00008000u) vr[i].w[e] &= 0xFFFF0000u;
                            if (f & 0x80000000u) vr[i].w[e] &= 0x0000FFFFu;
                        }
                }
            }
        }
        {
            typename Kd::VVec pf[RT][Kd::kp];
#pragma unroll
            for (int t = 0; t < RT; t++) split8<Kd::kp>(p[t], pf[t]);
#pragma unroll
            for (int i = 0; i < ND; i++) {
                const typename Kd::VVec v = widen<typename Kd::VVec>(vr[i]);
#pragma unroll
                for (int n = Kd::kp - 1; n >= 0; n--)
#pragma unroll
                    for (int t = 0; t < RT; t++) o[t][i] = mma(v, pf[t][n], o[t][i]);
            }
        }
        if constexpr (TYPE != SV_KV_I8) {
            if (odd) {
#pragma unroll 1
                for (int s = 0; s < kBlk; s++) {
                    const uint8_t *v = blk + (32 * D + ((s >> 3) * D + 4 * g) * 8 + (s & 7)) * ESZ;
#pragma unroll
                    for (int t = 0; t < RT; t++) {
                        float w = p[t][0];
#pragma unroll
                        for (int e = 1; e < 8; e++) w = (s & 7) == e ? p[t][e] : w;
                        const int from = 16 * (s >> 3) + col;
                        w = __shfl(w, from, 64);
                        const bool sees = __shfl(seen[t], from, 64) >> (s & 7) & 1u;
#pragma unroll
                        for (int i = 0; i < ND; i++)
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const uint32_t h = gld(reinterpret_cast<const uint16_t *>(v) + (16 * i + k) * 8);
                                if (!odd_pair<TYPE>(h) || !sees) continue;
                                const float y = TYPE == SV_KV_F16 ? half_bits_to_float(h) : __uint_as_float(h << 16);
                                o[t][i][k] += times_parts<Kd::kp, typename Kd::VVec>(w, y);
                            }
                    }
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (jn < last) load_v(blk_n);
        j = jn;
        page = page_n;
        blk = blk_n;
        jn = jnn;
        page_n = page_nn;
    }

    // ---- the waves' results joined: (0 + 2) + (1 + 3)
#pragma unroll
    for (int t = 0; t < RT; t++) {
        l[t] += __shfl_xor(l[t], 16, 64);
        l[t] += __shfl_xor(l[t], 32, 64);
        if (g == 0) {
            s_m[wave][16 * t + col] = mx[t];
            s_l[wave][16 * t + col] = l[t];
        }
    }
    __syncthreads();  // the queries are no longer read
#pragma unroll
    for (int t = 0; t < RT; t++) {
        float top = s_m[0][16 * t + col];
#pragma unroll
        for (int w = 1; w < kWaves; w++) top = fmaxf(top, s_m[w][16 * t + col]);
        const float by = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[t] - top);
#pragma unroll
        for (int i = 0; i < ND; i++) o[t][i] *= by;
        if (wave >= 2)
#pragma unroll
            for (int i = 0; i < ND; i++)
                *reinterpret_cast<f4 *>(s_o + ((wave - 2) * ROWS + 16 * t + col) * LD + 16 * i + 4 * g) = o[t][i];
    }
    __syncthreads();
    if (wave < 2) {
#pragma unroll
        for (int t = 0; t < RT; t++)
#pragma unroll
            for (int i = 0; i < ND; i++) {
                f4 *at = reinterpret_cast<f4 *>(s_o + (wave * ROWS + 16 * t + col) * LD + 16 * i + 4 * g);
                *at = o[t][i] + *at;
            }
    }
    __syncthreads();
    // ---- o = o0 + o1, l, m per row; out, or the chunk's part
    const int n = min(ROWS, rows - row0);
    const int64_t part = ((static_cast<int64_t>(b) * heads + head) * a.chunks + c) * a.rows + row0;
    for (int i = threadIdx.x; i < n * (D / 4); i += 64 * kWaves) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        f4 v = *reinterpret_cast<f4 *>(s_o + r * LD + d) + *reinterpret_cast<f4 *>(s_o + (ROWS + r) * LD + d);
        float top = s_m[0][r];
        for (int w = 1; w < kWaves; w++) top = fmaxf(top, s_m[w][r]);
        float sum = 0.0f;
        if (top != -INFINITY)
            for (int w = 0; w < kWaves; w++) sum += s_l[w][r] * __builtin_amdgcn_exp2f(s_m[w][r] - top);
        if (alone) {
            const bool over = a.max_len && sp.len + sp.n > a.max_len;
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
            v = over ? f4{NAN, NAN, NAN, NAN} : v * inv;
            *reinterpret_cast<f4 *>(s_o + r * LD + d) = v;
            if (over && i == 0) kv_flag(a.kv, SV_KV_OVER_MAX);
        } else {
            *(SV_GLOBAL f4 *)(a.part_o + (part + r) * D + d) = v;
            if (d == 0) {
                gst(a.part_m + part + r, top);
                gst(a.part_l + part + r, sum);
            }
        }
    }
    if (alone) {
        __syncthreads();
        finish_rows(a, s_o, LD, b, head, row0, n);
    }
}

template <int TYPE, int D>
static int launch_dim(const AttnArgs &a, int rt, dim3 grid, hipStream_t st) {
    if constexpr (D <= 128) {
        if (rt == 4) {
            hipLaunchKernelGGL((kv_attn_kernel<TYPE, D, 4>), grid, dim3(64 * kWaves), 0, st, a);
            return hip_check(hipGetLastError(), "kv_attention launch");
        }
        if (rt == 2) {
            hipLaunchKernelGGL((kv_attn_kernel<TYPE, D, 2>), grid, dim3(64 * kWaves), 0, st, a);
            return hip_check(hipGetLastError(), "kv_attention launch");
        }
    }
    hipLaunchKernelGGL((kv_attn_kernel<TYPE, D, 1>), grid, dim3(64 * kWaves), 0, st, a);
    return hip_check(hipGetLastError(), "kv_attention launch");
}

template <int TYPE>
static int launch_type(const AttnArgs &a, int rt, dim3 grid, hipStream_t st) {
    switch (a.kv.dim) {
        case 32: return launch_dim<TYPE, 32>(a, rt, grid, st);
        case 64: return launch_dim<TYPE, 64>(a, rt, grid, st);
        case 96: return launch_dim<TYPE, 96>(a, rt, grid, st);
        case 128: return launch_dim<TYPE, 128>(a, rt, grid, st);
        case 160: return launch_dim<TYPE, 160>(a, rt, grid, st);
        case 192: return launch_dim<TYPE, 192>(a, rt, grid, st);
        case 224: return launch_dim<TYPE, 224>(a, rt, grid, st);
        case 256: return launch_dim<TYPE, 256>(a, rt, grid, st);
    }
    return fail(SV_ERR_SHAPE, "kv_attention: unsupported head dimension");
}

#if SV_INST_KV == 1
int attn_launch_f16(const AttnArgs &a, int rt, dim3 grid, hipStream_t st) { return launch_type<SV_KV_F16>(a, rt, grid, st); }
#elif SV_INST_KV == 30
int attn_launch_bf16(const AttnArgs &a, int rt, dim3 grid, hipStream_t st) { return launch_type<SV_KV_BF16>(a, rt, grid, st); }
#else
int attn_launch_i8(const AttnArgs &a, int rt, dim3 grid, hipStream_t st) { return launch_type<SV_KV_I8>(a, rt, grid, st); }
#endif

}  // namespace sv
