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

__device__ __forceinline__ float xor16_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}

constexpr int kWaves = 4;

template <int TYPE, int D, int RT>
__global__ __launch_bounds__(64 * kWaves, 1) void kv_attn_kernel(AttnArgs a) {
    using Kd = Kind<TYPE>;
    constexpr int NC = D / 32, ND = D / 16, ESZ = Kd::esz;
    constexpr int LD = D + 4;
    constexpr int ROWS = 16 * RT;
    // the waves' results: o of two waves at a time, m and l of all
    __shared__ float s_o[2][ROWS][LD];
    __shared__ float s_m[kWaves][ROWS], s_l[kWaves][ROWS];

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
    const int sid = a.bt.seq ? gld(a.bt.seq + b) : b;
    if (sid < 0 || sid >= a.kv.seqs) return;
    const Span sp = span_of(a, b, sid);
    const int ac = chunk_of(sp, c);
    const bool alone = a.chunks == 1;  // no join: this workgroup finishes the rows
    if (ac >= sp.end && !alone) return;
    const int row0 = tile * ROWS;
    const int rows = sp.n * a.group;  // of this sequence, in use
    if (row0 >= rows) return;

    // ---- the rows' queries, as the second operand of S^T = K Q^T
    typename Kd::KVec qf[RT][NC][Kd::kq];
    float rs[RT];           // what the scores are multiplied by (a power of two)
    uint32_t mask[RT];      // the new rows that the row sees
    int64_t pos[RT];
#pragma unroll
    for (int t = 0; t < RT; t++) {
        const int r = row0 + 16 * t + col;
        const bool live = r < rows;
        const int m = live ? r / a.group : 0;
        const int hq = head * a.group + (live ? r % a.group : 0);
        mask[t] = live ? row_mask(a, b, m) : 0u;
        pos[t] = sp.len + row_depth(a, b, m);
        const float *qp = a.q + ((static_cast<int64_t>(b) * a.bt.M + m) * a.q_heads + hq) * D;
        float xq[NC][8];
        float top = 0.0f;
#pragma unroll
        for (int cc = 0; cc < NC; cc++) {
            const int d0 = 32 * cc + 8 * g;
            const uint4 u0 = gld16(qp + d0), u1 = gld16(qp + d0 + 4);
            const uint32_t u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
            for (int e = 0; e < 8; e++) xq[cc][e] = __uint_as_float(u[e]);
        }
        if (a.rope.mode != SV_ROPE_NONE) {
            const int half = a.rope.rot / 2;
            const int64_t at = pos[t] < a.rope.n_pos ? pos[t] : a.rope.n_pos - 1;
            const float *cs = a.rope.table + at * half * 2;
            const bool pairs = a.rope.mode == SV_ROPE_PAIRS;
#pragma unroll
            for (int cc = 0; cc < NC; cc++) {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int d = 32 * cc + 8 * g + e;
                    if (d >= a.rope.rot) continue;
                    const bool second = pairs ? e & 1 : d >= half;
                    const int p = pairs ? d >> 1 : (second ? d - half : d);
                    const float own = pairs ? 0.0f : xq[cc][e];
                    const float other = pairs ? 0.0f : gld(qp + (second ? d - half : d + half));
                    const float co = gld(cs + 2 * p), si = gld(cs + 2 * p + 1);
                    if (pairs) {
                        if (e & 1) continue;
                        const float x0 = xq[cc][e], x1 = xq[cc][e | 1];
                        xq[cc][e] = __fsub_rn(__fmul_rn(x0, co), __fmul_rn(x1, si));
                        xq[cc][e | 1] = __fadd_rn(__fmul_rn(x1, co), __fmul_rn(x0, si));
                    } else {
                        xq[cc][e] = second ? __fadd_rn(__fmul_rn(own, co), __fmul_rn(other, si))
                                           : __fsub_rn(__fmul_rn(own, co), __fmul_rn(other, si));
                    }
                }
            }
        }
#pragma unroll
        for (int cc = 0; cc < NC; cc++)
#pragma unroll
            for (int e = 0; e < 8; e++) {
                xq[cc][e] = live ? xq[cc][e] * a.scale : 0.0f;
                top = fmaxf(top, fabsf(xq[cc][e]));
            }
        rs[t] = 1.0f;
        if constexpr (__is_same(typename Kd::KVec, h8)) {
            // the row's largest magnitude into [2^12, 2^13)
            top = xor16_max(top);
            const int ex = static_cast<int>(__float_as_uint(top) >> 23);  // biased; 255 = not finite
            const int up = ex == 0 || ex == 255 ? 0 : max(-100, min(100, 12 - (ex - 127)));
            const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            rs[t] = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
            for (int cc = 0; cc < NC; cc++)
#pragma unroll
                for (int e = 0; e < 8; e++) xq[cc][e] *= by;
        }
#pragma unroll
        for (int cc = 0; cc < NC; cc++) split8<Kd::kq>(xq[cc], qf[t][cc]);
    }

    f4 o[RT][ND];
    float mx[RT], l[RT];
#pragma unroll
    for (int t = 0; t < RT; t++) {
        mx[t] = -INFINITY;
        l[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < ND; i++) o[t][i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // ---- the wave's blocks
    const int per = a.chunk / kBlk;
    int64_t j = static_cast<int64_t>(ac) * per + wave;
    const int64_t last = min(static_cast<int64_t>(ac + 1) * per, (sp.total + kBlk - 1) / kBlk);
    const int64_t whole = sp.len + sp.n - a.window;  // with a window: from here on every row's window has begun
    for (; j < last; j += kWaves) {
        const int64_t s0 = j * kBlk;
        if (s0 >= a.sinks && s0 + kBlk <= sp.lo) continue;  // between the sinks and every window
        const int page = kv_page_of(a.kv, sid, j >> a.kv.blk_shift);
        if (page < 0) continue;
        const uint8_t *blk = kv_block(a.kv, a.layer, page, head, static_cast<int>(j & ((1 << a.kv.blk_shift) - 1)));
        Raw<ESZ> kr[NC][2], vr[ND];
#pragma unroll
        for (int cc = 0; cc < NC; cc++)
#pragma unroll
            for (int u = 0; u < 2; u++)
                kr[cc][u] = load_raw<ESZ>(blk + (((cc * 4 + g) * 32) + 8 * (col >> 2) + 4 * u + (col & 3)) * 8 * ESZ);
#pragma unroll
        for (int i = 0; i < ND; i++) vr[i] = load_raw<ESZ>(blk + (32 * D + (g * D + 16 * i + col) * 8) * ESZ);
        float ks[8], vs[8];  // int8: the scales of the lane group's eight slots
        if constexpr (TYPE == SV_KV_I8) {
            const float *sc = reinterpret_cast<const float *>(blk + 64 * D) + 8 * g;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                ks[e] = gld(sc + e);
                vs[e] = gld(sc + 32 + e);
            }
        }
        const bool edge = s0 + kBlk > sp.len || (a.window && s0 < whole && s0 + kBlk > a.sinks);
        // slots of the lane group that any row of the tile sees, and those that all see
        uint32_t any_sees = 0xFFu, all_see = 0xFFu;
        if (edge) any_sees = 0u;
        float p[RT][8];
        uint32_t seen[RT];  // slots of the lane group that the lane's row sees
#pragma unroll
        for (int t = 0; t < RT; t++) {
            f4 acc[2];
            acc[0] = acc[1] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int cc = 0; cc < NC; cc++)
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int n = Kd::kq - 1; n >= 0; n--)
                        acc[u] = mma(widen<typename Kd::KVec>(kr[cc][u]), qf[t][cc][n], acc[u]);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                p[t][e] = acc[e >> 2][e & 3] * rs[t];
                if constexpr (TYPE == SV_KV_I8) p[t][e] *= ks[e];
            }
            seen[t] = 0xFFu;
            if (edge) {
                const bool live = row0 + 16 * t + col < rows;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int64_t slot = s0 + 8 * g + e;
                    const int nth = static_cast<int>(slot - sp.len);
                    bool sees = nth < 0 || (nth < sp.n && (mask[t] >> nth & 1u));
                    if (slot >= sp.total) sees = false;
                    if (a.window && sees) {
                        const int64_t kpos = nth < 0 ? slot : sp.len + row_depth(a, b, nth);
                        sees = pos[t] - kpos < a.window || kpos < a.sinks;
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
            float top = p[t][0];
#pragma unroll
            for (int e = 1; e < 8; e++) top = fmaxf(top, p[t][e]);
            const float now = fmaxf(mx[t], xor16_max(top));
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
        bool odd = false;
        if constexpr (TYPE != SV_KV_I8) {
            if (edge) {
                // Values in slots that no row sees count as 0, whatever they
                // hold.  Infinities and NaN in a slot that some rows see and
                // others do not cannot go through a product with weight 0:
                // they are taken out and added row by row.
                uint32_t keep2[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                    keep2[e] = (any_sees >> (2 * e) & 1u ? 0x0000FFFFu : 0u) | (any_sees >> (2 * e + 1) & 1u ? 0xFFFF0000u : 0u);
                uint32_t found = 0;
#pragma unroll
                for (int i = 0; i < ND; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        vr[i].w[e] &= keep2[e];
                        const uint32_t f = odd_pair<TYPE>(vr[i].w[e]);
                        found |= f & ((all_see >> (2 * e) & 1u ? 0u : 0x00008000u) | (all_see >> (2 * e + 1) & 1u ? 0u : 0x80000000u));
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
#pragma unroll
        for (int t = 0; t < RT; t++) {
            typename Kd::VVec pf[Kd::kp];
            split8<Kd::kp>(p[t], pf);
#pragma unroll
            for (int i = 0; i < ND; i++)
#pragma unroll
                for (int n = Kd::kp - 1; n >= 0; n--)
                    o[t][i] = mma(widen<typename Kd::VVec>(vr[i]), pf[n], o[t][i]);
        }
        if constexpr (TYPE != SV_KV_I8) {
            if (odd) {
                for (int gg = 0; gg < 4; gg++) {
#pragma unroll
                    for (int t = 0; t < RT; t++) {
                        const uint32_t sees = __shfl(seen[t], 16 * gg + col, 64);
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const float w = __shfl(p[t][e], 16 * gg + col, 64);
                            const uint8_t *v = blk + (32 * D + (gg * D + 4 * g) * 8 + e) * ESZ;
#pragma unroll
                            for (int i = 0; i < ND; i++)
#pragma unroll
                                for (int k = 0; k < 4; k++) {
                                    const uint32_t h = gld(reinterpret_cast<const uint16_t *>(v) + (16 * i + k) * 8);
                                    if (!odd_pair<TYPE>(h) || !(sees >> e & 1u)) continue;
                                    const float y = TYPE == SV_KV_F16 ? half_bits_to_float(h) : __uint_as_float(h << 16);
                                    o[t][i][k] += times_parts<Kd::kp, typename Kd::VVec>(w, y);
                                }
                        }
                    }
                }
            }
        }
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
    __syncthreads();
    float by[RT];
#pragma unroll
    for (int t = 0; t < RT; t++) {
        float top = s_m[0][16 * t + col];
#pragma unroll
        for (int w = 1; w < kWaves; w++) top = fmaxf(top, s_m[w][16 * t + col]);
        by[t] = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[t] - top);
#pragma unroll
        for (int i = 0; i < ND; i++) o[t][i] *= by[t];
        if (wave >= 2)
#pragma unroll
            for (int i = 0; i < ND; i++) *reinterpret_cast<f4 *>(&s_o[wave - 2][16 * t + col][16 * i + 4 * g]) = o[t][i];
    }
    __syncthreads();
    if (wave < 2) {
#pragma unroll
        for (int t = 0; t < RT; t++)
#pragma unroll
            for (int i = 0; i < ND; i++) {
                f4 *at = reinterpret_cast<f4 *>(&s_o[wave][16 * t + col][16 * i + 4 * g]);
                *at = o[t][i] + *at;
            }
    }
    __syncthreads();
    // ---- o = o0 + o1, l, m per row; out, or the chunk's part
    const int n = min(ROWS, rows - row0);
    const int64_t part = ((static_cast<int64_t>(b) * heads + head) * a.chunks + c) * a.rows + row0;
    for (int i = threadIdx.x; i < n * (D / 4); i += 64 * kWaves) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        f4 v = *reinterpret_cast<f4 *>(&s_o[0][r][d]) + *reinterpret_cast<f4 *>(&s_o[1][r][d]);
        float top = s_m[0][r];
        for (int w = 1; w < kWaves; w++) top = fmaxf(top, s_m[w][r]);
        float sum = 0.0f;
        if (top != -INFINITY)
            for (int w = 0; w < kWaves; w++) sum += s_l[w][r] * __builtin_amdgcn_exp2f(s_m[w][r] - top);
        if (alone) {
            const bool over = a.max_len && sp.len + sp.n > a.max_len;
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
            v = over ? f4{NAN, NAN, NAN, NAN} : v * inv;
            *reinterpret_cast<f4 *>(&s_o[0][r][d]) = v;
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
        finish_rows(a, &s_o[0][0][0], LD, n, [&](int i) -> int64_t {
            const int r = row0 + i;
            return (static_cast<int64_t>(b) * a.bt.M + r / a.group) * a.q_heads + head * a.group + r % a.group;
        });
    }
}

template <int TYPE, int D>
static int launch_dim(const AttnArgs &a, int rt, dim3 grid, hipStream_t st) {
    if constexpr (D <= 128) {
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
