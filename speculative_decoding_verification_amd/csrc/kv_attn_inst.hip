// kv_attn_inst.hip - attention of the new rows over the cache, one chunk of
// the length per workgroup; compiled once per cache type (SV_INST_KV).
//
// For a row with query q and the visible slots j of a chunk:
//   s_j = q . k_j,  m = max s_j,  l = sum 2^(s_j - m),  o = sum 2^(s_j - m) v_j
// in one pass over the chunk with a running m, l and o (q is scaled by
// scale * log2(e) first).  The rows of one key head, M * group of them, are
// the 16 columns of a tile; a wave takes every W-th block of 32 slots:
//   S^T [32 slots x 16 rows] = K Q^T    two 16x16x32 products per 32 of dim
//   O^T [dim x 16 rows] += V^T P^T      one 16x16x32 product per 16 of dim
// Row r of the first product's tile t is slot 8 (r / 4) + 4 t + r % 4, so
// lane group g (lanes 16 g ..) holds the scores of slots 8 g .. 8 g + 7, and
// these are the eight it supplies to the second product: the weights stay
// where they are, and a block's keys and values are the products' operands
// as they lie, 16 (int8: 8) contiguous bytes a lane.
//
// Precision: the fp32 q and weights enter as sums of parts, two for fp16 (q
// scaled by a power of two per row, the weights by 2^15, so that the second
// part stays a normal number) and three for bf16.  Three bf16 parts are exact.
// The first fp16 part leaves a whole number of at most 2^12 steps of fp32, and
// the second takes all of it but, in a quarter of the values, the last step: a
// factor is at most 2^-23 off, as after one rounding more of fp32.  A third
// part would be exact and costs registers and half as many products again
// (us: 5 x 4099 slots 17.2 against 18.8, trees 24.6 against 36.7, wide window
// 124 against 155, int8 batch 80.5 against 89.6); the outputs of all measured
// cases are closer to 64 bits than those of plain fp32 sums without it.  int8 codes are exact in
// fp16 and go with it; there a weight carries its value's scale d_j, and m is
// the maximum of s_j + log2 d_j, so that the weights end at 1 whatever the
// scales are (scales below 2^-80 count as that in m: sums of such values
// alone keep fewer bits).  Scores beyond 2^24 in base 2 leave no room in m for
// the 2^15 or the scale; such rows go without them (see kExact), int8 ones
// through an fp32 path of their own.
//
// Bound by memory for long caches: a block of 32 slots is 128 dim bytes (64
// dim for int8) and is read once.  Each wave keeps the next blocks on their
// way in a ring of its own in LDS, filled by loads that go there directly, so
// that what is in flight costs no registers; the ring's halves (a block's
// keys, its values) are refilled as soon as they are in registers.  Measured
// with the join, heads of 128 and groups of 5, a read alone reaching 7.1 TB/s:
//   131001 slots of 8 heads, 5 rows, bf16    537 MB in 95 us, 5.7 TB/s
//   32 windows of 4096, 5 rows, fp16         523 MB in 124 us, 4.2 TB/s: the
//     last, partly filled round of workgroups
//   16 sequences up to 16384, int8           284 MB in 80 us, 3.5 TB/s: the
//     same (on average 1.3 of the two waves a SIMD are there), and waits: the
//     SIMDs issue vector instructions (600 a block and wave, 64 of them matrix
//     ones) in 45 % of the time, their matrix units are busy in 18 %, and a
//     wave waits for loads and barriers in 29 % of its own
// Short calls are bound by latency: of 13.5 us for 4099 slots about 5 go by
// before a wave has its first block (lengths, page, queries, angles), 3 for
// its blocks and 3 for the sums of the waves.
#include <atomic>
#include <type_traits>

#include "kv_attn.h"

namespace sv {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
#define SV_LDS __attribute__((address_space(3)))

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
    typedef h8 VVec;
    static constexpr int kq = 2, kp = 2, esz = 1;
};

constexpr float kLeastScale = -80.0f;
// Whole numbers up to here stay exact with 15 taken off.
constexpr float kExact = 16777200.0f;  // 2^24 - 16

__device__ __forceinline__ f4 mma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f4 mma(b8 a, b8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// x = sum of N parts of the narrow type, each the rounding of what is left
// (fp16: taken off by the instruction that reads halves as they are).
template <int N, typename V8>
__device__ __forceinline__ void split8(const float (&x)[8], V8 (&part)[N]) {
    typedef decltype(part[0][0] + part[0][0]) E;
    typedef E E2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        f2 left = {x[e], x[e + 1]};
#pragma unroll
        for (int n = 0; n < N; n++) {
            const E2 h = __builtin_convertvector(left, E2);
            part[n][e] = h.x;
            part[n][e + 1] = h.y;
            if (n + 1 == N) break;
            if constexpr (__is_same(E, _Float16)) {
                uint32_t u;
                __builtin_memcpy(&u, &h, 4);
                float x0, x1;
                asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(x0) : "v"(u), "v"(left.x));
                asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(x1) : "v"(u), "v"(left.y));
                left = f2{x0, x1};
            } else {
                uint32_t u;
                __builtin_memcpy(&u, &h, 4);
                left.x -= __uint_as_float(u << 16);
                left.y -= __uint_as_float(u & 0xFFFF0000u);
            }
        }
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

// Raw piece of a block as one lane holds it.
template <int ESZ>
struct Raw {
    uint32_t w[2 * ESZ];
};

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
    return v;
}

// An element pair's bits that make it an infinity or NaN.
template <int TYPE>
__device__ __forceinline__ uint32_t odd_pair(uint32_t w) {
    return ((w & 0x7FFF7FFFu) + (TYPE == SV_KV_F16 ? 0x04000400u : 0x00800080u)) & 0x80008000u;
}

// Largest value and sum over the four lanes that share a row (16 and 32 lanes
// apart).
__device__ __forceinline__ float row_max(float v) {
    float a, b;
    swap16(v, &a, &b);
    swap32(fmaxf(a, b), &a, &b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float row_sum(float v) {
    float a, b;
    swap16(v, &a, &b);
    swap32(a + b, &a, &b);
    return a + b;
}

// ------------------------------------------------------------- the ring
// Pieces of a ring half into registers, behind a wait that leaves the last
// LEAVE transfers of the wave on their way: the waits are in the same asm
// block as the reads, so nothing is taken for loaded before it is.
template <int LEAVE, int STRIDE, int N, int FROM = 0>
__device__ __forceinline__ void ring_read(uint32_t at, Raw<2> *r) {
    u32x4 v[8];
    if constexpr (N >= 8) {
        asm volatile(
            "s_waitcnt vmcnt(%17)\n"
            "ds_read_b128 %0, %8 offset:%9\n ds_read_b128 %1, %8 offset:%10\n"
            "ds_read_b128 %2, %8 offset:%11\n ds_read_b128 %3, %8 offset:%12\n"
            "ds_read_b128 %4, %8 offset:%13\n ds_read_b128 %5, %8 offset:%14\n"
            "ds_read_b128 %6, %8 offset:%15\n ds_read_b128 %7, %8 offset:%16\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
            : "v"(at), "n"(FROM), "n"(FROM + STRIDE), "n"(FROM + 2 * STRIDE), "n"(FROM + 3 * STRIDE),
              "n"(FROM + 4 * STRIDE), "n"(FROM + 5 * STRIDE), "n"(FROM + 6 * STRIDE), "n"(FROM + 7 * STRIDE), "n"(LEAVE)
            : "memory");
    } else if constexpr (N >= 4) {
        asm volatile(
            "s_waitcnt vmcnt(%9)\n"
            "ds_read_b128 %0, %4 offset:%5\n ds_read_b128 %1, %4 offset:%6\n"
            "ds_read_b128 %2, %4 offset:%7\n ds_read_b128 %3, %4 offset:%8\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
            : "v"(at), "n"(FROM), "n"(FROM + STRIDE), "n"(FROM + 2 * STRIDE), "n"(FROM + 3 * STRIDE), "n"(LEAVE)
            : "memory");
    } else {
        asm volatile(
            "s_waitcnt vmcnt(%5)\n"
            "ds_read_b128 %0, %2 offset:%3\n ds_read_b128 %1, %2 offset:%4\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0]), "=&v"(v[1])
            : "v"(at), "n"(FROM), "n"(FROM + STRIDE), "n"(LEAVE)
            : "memory");
    }
    constexpr int T = N >= 8 ? 8 : N >= 4 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < T; i++) {
        r[i].w[0] = v[i].x;
        r[i].w[1] = v[i].y;
        r[i].w[2] = v[i].z;
        r[i].w[3] = v[i].w;
    }
    if constexpr (N > T) ring_read<LEAVE, STRIDE, N - T, FROM + T * STRIDE>(at, r + T);
}
// int8: pieces of 8 bytes; pairs of them STRIDE apart, the second EVERY past
// the first (keys: the two slots of a piece's tiles), or EVERY = 0.
template <int LEAVE, int STRIDE, int EVERY, int N, int FROM = 0>
__device__ __forceinline__ void ring_read(uint32_t at, Raw<1> *r) {
    u32x2 v[4];
    constexpr int O1 = EVERY ? FROM + EVERY : FROM + STRIDE, O2 = EVERY ? FROM + STRIDE : FROM + 2 * STRIDE;
    constexpr int O3 = EVERY ? O2 + EVERY : FROM + 3 * STRIDE;
    if constexpr (N >= 4) {
        asm volatile(
            "s_waitcnt vmcnt(%9)\n"
            "ds_read_b64 %0, %4 offset:%5\n ds_read_b64 %1, %4 offset:%6\n"
            "ds_read_b64 %2, %4 offset:%7\n ds_read_b64 %3, %4 offset:%8\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
            : "v"(at), "n"(FROM), "n"(O1), "n"(O2), "n"(O3), "n"(LEAVE)
            : "memory");
    } else {
        asm volatile(
            "s_waitcnt vmcnt(%5)\n"
            "ds_read_b64 %0, %2 offset:%3\n ds_read_b64 %1, %2 offset:%4\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0]), "=&v"(v[1])
            : "v"(at), "n"(FROM), "n"(O1), "n"(LEAVE)
            : "memory");
    }
    constexpr int T = N >= 4 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < T; i++) {
        r[i].w[0] = v[i].x;
        r[i].w[1] = v[i].y;
    }
    constexpr int NEXT = EVERY ? FROM + T / 2 * STRIDE : FROM + T * STRIDE;
    if constexpr (N > T) ring_read<LEAVE, STRIDE, EVERY, N - T, NEXT>(at, r + T);
}
__device__ __forceinline__ void lds_read8(uint32_t at, uint32_t at4, float (&s)[8]) {
    u32x4 a, b;
    asm volatile("ds_read_b128 %0, %2\n ds_read_b128 %1, %3\n s_waitcnt lgkmcnt(0)"
                 : "=&v"(a), "=&v"(b)
                 : "v"(at), "v"(at4)
                 : "memory");
#pragma unroll
    for (int e = 0; e < 4; e++) {
        s[e] = __uint_as_float(a[e]);
        s[4 + e] = __uint_as_float(b[e]);
    }
}
// Transfers global memory to LDS, 16 bytes a lane (lane i to `to` + 16 i).
// ONCE: no other workgroup of the launch reads it, so it need not stay in
// the caches (non-temporal).
// OFFSET is added to both addresses by the instruction.
template <bool ONCE, int OFFSET = 0>
__device__ __forceinline__ void to_lds(const uint8_t *from, uint32_t to) {
    __builtin_amdgcn_global_load_lds(from, (SV_LDS void *)static_cast<uintptr_t>(to), 16, OFFSET, ONCE ? 2 : 0);
}
// Transfers I .. N - 1 of a half, 1024 bytes apart in LDS and in memory
// PAIR * (i / 2) + ODD * (i % 2) bytes from the lane's first, `own` bytes past a
// uniform address.  Four KB of memory share an address: the rest is the
// instruction's offset, which the LDS address takes back.  (An address in vector
// registers for each transfer takes an addition and two scalar registers for its
// constant, of which the loop has too few: us, 16 rounds over 32768 shared
// slots 140.5 against 138.5, trees 25.5 against 25.2.)
template <bool ONCE, int PAIR, int ODD, int N, int I = 0>
__device__ __forceinline__ void half_to_lds(const uint8_t *from, uint32_t own, uint32_t to) {
    constexpr int AT = PAIR * (I / 2) + ODD * (I % 2), OFFSET = AT % 4096;
    static_assert(I * 1024 >= OFFSET, "an LDS address below the half");
    to_lds<ONCE, OFFSET>(from + (AT - OFFSET) + own, to + I * 1024 - OFFSET);
    if constexpr (I + 1 < N) half_to_lds<ONCE, PAIR, ODD, N, I + 1>(from, own, to);
}

// Waves and their rings, for two workgroups a compute unit: four where the
// registers of two waves fit a SIMD (int8, and fp16 up to 128: bf16's queries
// take half as much again), else two.  A function of the type and dim alone:
// the waves share a chunk's blocks, so a row's sums depend on it.  (fp16 with
// two: trees of up to 8191 slots 35 against 28 us, 32 windows of 4096 142
// against 134; all waves in one workgroup: 5 x 4099 slots 19.6 against 18.2,
// a single row's 300 slots 9.1 against 9.5.)  A ring holds one block, or 8 KB
// of smaller ones: with more on its way a load only waits longer behind the
// others (16 KB for int8 and 32 KB for bf16: window of 1024 17.0 against 16.2
// us, int8 batch 81.7 against 79.7).
template <int TYPE, int D, int RT>
struct Shape {
    using Kd = Kind<TYPE>;
    static constexpr bool TWO = TYPE == SV_KV_I8 || (TYPE == SV_KV_F16 && D <= 128);
    static constexpr int W = TWO ? 4 : 2;                       // waves
    static constexpr int HALF = 32 * D * Kd::esz;               // bytes of a block's keys, or values
    static constexpr int LOADS = HALF / 1024;                   // transfers of a half
    static constexpr int SCALES = TYPE == SV_KV_I8 ? 1 : 0;     // and one of both scales with the keys
    // halves of a wave's ring, at least a block
    static constexpr int FIT = 8192 / HALF / 2 * 2;
    static constexpr int N = FIT < 2 ? 2 : FIT > 8 ? 8 : FIT;
    // [half][wave], then the scales [block][wave]
    static constexpr int SCALES_AT = N * W * HALF, RING_BYTES = SCALES_AT + N / 2 * W * 256 * SCALES;
    // transfers that may still be on their way when the oldest half is read:
    // those of the halves after it
    static constexpr int LEAVE_K = (N / 2 - 1) * (LOADS + SCALES) + N / 2 * LOADS;
    static constexpr int LEAVE_V = N / 2 * (LOADS + SCALES) + (N / 2 - 1) * LOADS;
    static_assert(LEAVE_K < 64 && LEAVE_V < 64, "the wait counter has six bits");
    static constexpr int ROWS = 16 * RT, LD = D + 4;
    // The fp32 rows that the queries are made of, and the angles of up to 16
    // positions.  EARLY: behind the first keys, which are requested before
    // they are used, or behind the scales; else in the ring's beginning.  (us,
    // early against late: 5 x 4099 slots 17.3 against 17.8, trees 24.7 against
    // 25.3, window of 4096 123.6 against 125; two waves a workgroup, 5 x
    // 131001 slots 96.5 against 94.3; one tile of rows, 300 slots 9.9 against
    // 9.7.)
    static constexpr int ROWS_BYTES = ROWS * D * 4, BYTES = ROWS_BYTES + 16 * D * 4;
    static constexpr int AT = !SCALES || W * HALF + BYTES <= SCALES_AT ? W * HALF : RING_BYTES;
    static constexpr bool EARLY = TWO && RT > 1 && AT + BYTES <= kMaxLds - 2048;
    static constexpr int STAGED = EARLY ? AT : 0, ANGLES = STAGED + ROWS_BYTES, STAGED_END = STAGED + BYTES;
    static constexpr int SUMS = W * ROWS * LD * 4;              // the waves' sums, after the blocks
    static constexpr int MOST = RING_BYTES > SUMS ? RING_BYTES : SUMS, LDS = MOST > STAGED_END ? MOST : STAGED_END;
};

// Queries are staged as they lie, a row's quads of four elements exchanged by
// the row's number, so that reads of one quad of 16 rows spread over the
// banks: quad q of row i is the row's (q ^ i % 8)-th.
template <int D>
__device__ __forceinline__ uint32_t quad_at(uint32_t staged, int i, int q) {
    return staged + (i * (D / 4) + (q ^ (i & 7))) * 16;
}
__device__ __forceinline__ const float *query_of(const AttnArgs &a, int b, int head, int r) {
    const int m = a.by_group(r);
    return a.q + ((static_cast<int64_t>(b) * a.bt.M + m) * a.q_heads + head * a.group + (r - m * a.group)) * a.kv.dim;
}

// Position of new row m of sequence b, whose length is `len`.
__device__ __forceinline__ int place_of(const AttnArgs &a, int len, int b, int m) {
    return len + (a.bt.tree ? __popc(row_mask(a, b, m) & ((1u << m) - 1)) : m);
}
// The same where sequences share chunks: rows m are numbered through all
// sequences (b and len are not used).
__device__ __forceinline__ int place_of(const AttnShared &a, int, int, int m) {
    const int b = a.by_m(m), sid = a.bt.seq ? gld(a.bt.seq + b) : b;
    const int len = sid >= 0 && sid < a.kv.seqs ? static_cast<int>(kv_len_of(a.kv, sid)) : 0;
    return place_of(static_cast<const AttnArgs &>(a), len, b, m - b * a.bt.M);
}

// Positions whose angles are staged: as many as one sequence has rows.  Tiles
// of several sequences' rows may have more; then they are read where they are.
__device__ __forceinline__ bool angles_staged(const AttnArgs &a, int row0, int n) {
    return a.rope.rot % 8 == 0 && a.by_group(row0 + n - 1) - a.by_group(row0) < SV_MAX_M;
}

// Requests n rows' queries and, unless a rotation's quads of pairs are not
// whole, the angles of their positions [position][rot].
template <int D, int W, typename Args>
__device__ __forceinline__ void stage_rows(const Args &a, int len, int b, int head, int row0, int n, int wave,
                                           uint32_t staged, uint32_t angles) {
    const int lane = threadIdx.x & 63;
    if (a.rope.mode != SV_ROPE_NONE && angles_staged(a, row0, n)) {
        const int m0 = a.by_group(row0), of = a.by_group(row0 + n - 1) - m0 + 1;
        int at = 0;
        if (lane < of) at = place_of(a, len, b, m0 + lane);
        for (int i = wave; i < of; i += W) {
            const int pos = min(__builtin_amdgcn_readlane(at, i), a.rope.n_pos - 1);
            if (lane < a.rope.rot / 4)
                to_lds<false>(reinterpret_cast<const uint8_t *>(a.rope.table + static_cast<int64_t>(pos) * a.rope.rot + 4 * lane),
                              angles + i * a.rope.rot * 4);
        }
    }
    constexpr int QUADS = D / 4;
#pragma unroll 1
    for (int at = wave * 64; at < n * QUADS; at += W * 64) {
        const int i = (at + lane) / QUADS, q = ((at + lane) % QUADS) ^ (i & 7);
        to_lds<false>(reinterpret_cast<const uint8_t *>(query_of(a, b, head, row0 + min(i, n - 1)) + 4 * q),
                      staged + at * 16);
    }
}

// Turns the staged rows by their angles, four pairs a thread and step.
template <int D, int THREADS, typename Args>
__device__ __forceinline__ void turn_rows(const Args &a, int len, int b, int row0, int n, uint32_t staged,
                                          uint32_t angles) {
    const int rot = a.rope.rot, m0 = a.by_group(row0);
    if (!angles_staged(a, row0, n)) {  // pair by pair, with the angles where they are
        for (int it = threadIdx.x; it < n * (rot / 2); it += THREADS) {
            const int i = it / (rot / 2), p = it - i * (rot / 2);
            const int pos = place_of(a, len, b, a.by_group(row0 + i));
            const float *cs = a.rope.table + static_cast<int64_t>(min(pos, a.rope.n_pos - 1)) * rot + 2 * p;
            const int e0 = a.rope.mode == SV_ROPE_PAIRS ? 2 * p : p, e1 = a.rope.mode == SV_ROPE_PAIRS ? e0 + 1 : p + rot / 2;
            SV_LDS float *x0 = (SV_LDS float *)static_cast<uintptr_t>(quad_at<D>(staged, i, e0 / 4) + e0 % 4 * 4);
            SV_LDS float *x1 = (SV_LDS float *)static_cast<uintptr_t>(quad_at<D>(staged, i, e1 / 4) + e1 % 4 * 4);
            const float co = gld(cs), si = gld(cs + 1), u = *x0, v = *x1;
            *x0 = __fsub_rn(__fmul_rn(u, co), __fmul_rn(v, si));
            *x1 = __fadd_rn(__fmul_rn(v, co), __fmul_rn(u, si));
        }
        return;
    }
    const bool pairs = a.rope.mode == SV_ROPE_PAIRS;
    const int of = rot / 8;
#pragma unroll 1
    for (int it = threadIdx.x; it < n * of; it += THREADS) {
        const int i = a.by_turns(it), k = it - i * of;
        const uint32_t at0 = quad_at<D>(staged, i, pairs ? 2 * k : k), at1 = quad_at<D>(staged, i, pairs ? 2 * k + 1 : k + of);
        const uint32_t cs = angles + ((a.by_group(row0 + i) - m0) * rot + 8 * k) * 4;
        f4 x, y, c0, c1;
        asm volatile("ds_read_b128 %0, %4\n ds_read_b128 %1, %5\n ds_read_b128 %2, %6\n ds_read_b128 %3, %6 offset:16\n"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(x), "=&v"(y), "=&v"(c0), "=&v"(c1)
                     : "v"(at0), "v"(at1), "v"(cs)
                     : "memory");
        const f4 u = pairs ? f4{x.x, x.z, y.x, y.z} : x, v = pairs ? f4{x.y, x.w, y.y, y.w} : y;
        const f4 co = {c0.x, c0.z, c1.x, c1.z}, si = {c0.y, c0.w, c1.y, c1.w};
        f4 s, t;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            s[e] = __fsub_rn(__fmul_rn(u[e], co[e]), __fmul_rn(v[e], si[e]));
            t[e] = __fadd_rn(__fmul_rn(v[e], co[e]), __fmul_rn(u[e], si[e]));
        }
        x = pairs ? f4{s.x, t.x, s.y, t.y} : s;
        y = pairs ? f4{s.z, t.z, s.w, t.w} : t;
        asm volatile("ds_write_b128 %0, %2\n ds_write_b128 %1, %3" ::"v"(at0), "v"(at1), "v"(x), "v"(y) : "memory");
    }
}

// The queries of a row tile as the second operand of S^T = K Q^T, from the n
// staged rows (by reads in asm: the ring's transfers are on their way; lanes
// past the last row take that one), for fp16 multiplied by the power of two
// that brings the row's largest magnitude into [2^12, 2^13); the row's scores
// are multiplied by the returned power of two to undo that.
template <int TYPE, int D>
__device__ __forceinline__ float take_queries(uint32_t staged, int from, int n, float scale,
                                              typename Kind<TYPE>::KVec (&qf)[D / 32][Kind<TYPE>::kq]) {
    using Kd = Kind<TYPE>;
    constexpr int NC = D / 32;
    const int lane = threadIdx.x & 63, i = min(from + (lane & 15), n - 1), g = lane >> 4;
    const uint32_t at0 = quad_at<D>(staged, i, 2 * g), at1 = quad_at<D>(staged, i, 2 * g + 1);
    float x[NC][8];
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; c++) {
        lds_read8(at0 + 128 * c, at1 + 128 * c, x[c]);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            x[c][e] *= scale;
            top = fmaxf(top, fabsf(x[c][e]));
        }
    }
    float back = 1.0f;
    if constexpr (__is_same(typename Kd::KVec, h8)) {
        top = row_max(top);
        const int ex = static_cast<int>(__float_as_uint(top) >> 23);  // biased; 255 = not finite
        // -115 at least, so that both powers are normal numbers
        const int up = ex == 0 || ex == 255 ? 0 : min(100, 12 - (ex - 127));
        const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
        for (int c = 0; c < NC; c++)
#pragma unroll
            for (int e = 0; e < 8; e++) x[c][e] *= by;
    }
#pragma unroll
    for (int c = 0; c < NC; c++) split8<Kd::kq>(x[c], qf[c]);
    return back;
}

// The sequence, head and chunk of number u.  B lengths are read by the lanes,
// so that no workgroup is spent on a chunk that the longest sequence has and
// another has not.  The sinks' chunks, of few slots, come after all others:
// they fill the last round.
struct Unit {
    int b, head, c;  // b = -1 past the last
};
// With `skip` chunks shared, u counts only those after them.
__device__ __forceinline__ Unit find_unit(const AttnArgs &a, int u, int skip) {
    const int lane = threadIdx.x & 63;
    int passed = 0;
    for (int sinks = 0; sinks <= (a.sinks ? 1 : 0); sinks++)
        for (int b0 = 0; b0 < a.bt.B; b0 += 64) {
            const int b = b0 + lane;
            int own = 0, first = 0;
            if (b < a.bt.B) {
                const int sid = a.bt.seq ? gld(a.bt.seq + b) : b;
                if (sid >= 0 && sid < a.kv.seqs) {
                    const int n = kv_rows_of(a.bt.n_new, b, a.bt.M);
                    if (n) {
                        const Span sp = span_of(a, static_cast<int>(kv_len_of(a.kv, sid)), n);
                        const int chunks = chunks_of(a, sp);
                        first = min(sp.first + skip, chunks);
                        own = sinks ? first : chunks - first;
                    }
                }
            }
            const int upto = scan64(own * a.kv.heads), all = __builtin_amdgcn_readlane(upto, 63);
            if (passed + all > u) {
                const int at = __ffsll(__ballot(passed + upto > u)) - 1;
                const int n = __builtin_amdgcn_readlane(own, at);
                const int i = u - passed - __builtin_amdgcn_readlane(upto, at) + n * a.kv.heads, head = i / n;
                return Unit{b0 + at, head, i - head * n + (sinks ? 0 : __builtin_amdgcn_readlane(first, at))};
            }
            passed += all;
        }
    return Unit{-1, 0, 0};
}

__device__ __forceinline__ int shared_of(const AttnArgs &) { return 0; }
__device__ __forceinline__ int shared_of(const AttnShared &a) { return a.shared; }
__device__ __forceinline__ int shared_tiles_of(const AttnArgs &a) { return a.tiles; }
__device__ __forceinline__ int shared_tiles_of(const AttnShared &a) { return a.shared_tiles; }
__device__ __forceinline__ int by_shared_tiles(const AttnArgs &a, int x) { return a.by_tiles(x); }
__device__ __forceinline__ int by_shared_tiles(const AttnShared &a, int x) { return a.by_shared_tiles(x); }

// Marks the sequences of a tile's rows that do not hold chunk c as `sid`
// does: another page, none, or fewer committed slots.  Their rows' results
// are NaN, and the status says so.
__device__ __forceinline__ void find_strangers(const AttnShared &a, int sid, bool named, int c, int row0, int n,
                                               int threads, int *s_bad) {
    const int b0 = a.by_rows(row0), of = a.by_rows(row0 + n - 1) - b0 + 1;
    const int e0 = c * a.chunk >> a.kv.page_shift, entries = (((c + 1) * a.chunk - 1) >> a.kv.page_shift) - e0 + 1;
    for (int it = threadIdx.x; it < of * entries; it += threads) {
        const int i = it / entries, e = e0 + it - i * entries, b = b0 + i;
        const int own = a.bt.seq ? gld(a.bt.seq + b) : b;
        if (own < 0 || own >= a.kv.seqs || kv_rows_of(a.bt.n_new, b, a.bt.M) == 0) continue;
        const int page = kv_page_of(a.kv, own, e);
        if (named && page >= 0 && page == kv_page_of(a.kv, sid, e) && kv_len_of(a.kv, own) >= (c + 1) * a.chunk) continue;
        s_bad[i] = 1;
        kv_flag(a.kv, SV_KV_NOT_SHARED);
    }
}

// Args: AttnArgs, or AttnShared where the sequences share their first chunks.
// These are taken once for the rows of all sequences, 16 RT of them a
// workgroup, in the same way as a sequence's own: a row's bits are those of
// the call that does not share.
template <int TYPE, int D, int RT, typename Args>
__global__ __launch_bounds__((64 * Shape<TYPE, D, RT>::W), (Shape<TYPE, D, RT>::TWO ? 2 : 1)) void kv_attn_kernel(
    Args a) {
    using Kd = Kind<TYPE>;
    using S = Shape<TYPE, D, RT>;
    constexpr bool SHARED = __is_same(Args, AttnShared);
    fetch_args<sizeof(Args)>();
    constexpr int NC = D / 32, ND = D / 16, ESZ = Kd::esz, W = S::W, LD = S::LD, ROWS = S::ROWS;
    // Read past the caches.  Meant for blocks that one row group reads, which
    // dim and row tiles do not quite say: from 33 rows on, dims of 96 and 128
    // have several groups, whose second reading the placement below would let
    // L2 serve (80 rows of 128 over 8191 slots take 38 us), and up to 64 rows of
    // at most 64 are one.
    constexpr bool ONCE = D <= 128 && RT < 4 && !SHARED;
    extern __shared__ __align__(1024) uint8_t s_mem[];
    __shared__ float s_m[W][ROWS], s_l[W][ROWS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int heads = a.kv.heads;
    // Row groups of one chunk read the same blocks: eight workgroups apart,
    // so that the same XCD takes them and its L2 serves the second reading.
    int x = blockIdx.x;
    bool all = false;  // a shared chunk: rows of all sequences
    if constexpr (SHARED) {
        all = x < a.shared_grid;
        if (!all) x -= a.shared_grid;
    }
    const int tiles = SHARED && all ? shared_tiles_of(a) : a.tiles;
    const int u8 = SHARED && all ? by_shared_tiles(a, x / 8) : a.by_tiles(x / 8), tile = x / 8 - u8 * tiles, u = u8 * 8 + x % 8;
    const bool alone = !SHARED && a.chunks == 1;  // no join: this workgroup finishes the rows
    Unit unit;
    if (alone) {
        unit.b = a.by_heads(u);
        unit.head = u - unit.b * heads;
        unit.c = 0;
    } else if (SHARED && all) {
        unit.c = a.by_heads(u);
        unit.head = u - unit.c * heads;
        unit.b = 0;
        if (unit.c >= shared_of(a)) return;
    } else {
        unit = find_unit(a, u, shared_of(a));
        if (unit.b < 0) return;
    }
    const int b = unit.b, head = unit.head, c = unit.c;
    if (b >= a.bt.B) return;
    // a shared chunk's pages are those of the call's first sequence
    int sid = a.bt.seq ? __builtin_amdgcn_readfirstlane(gld(a.bt.seq + b)) : b;
    const bool named = sid >= 0 && sid < a.kv.seqs;
    if (!named) {
        if (!all) return;
        sid = 0;
    }
    const int len = __builtin_amdgcn_readfirstlane(static_cast<int>(kv_len_of(a.kv, sid)));
    Span sp = span_of(a, len, __builtin_amdgcn_readfirstlane(kv_rows_of(a.bt.n_new, b, a.bt.M)));
    const int row0 = tile * ROWS;
    int rows = sp.n * a.group;  // of this sequence, in use
    if (SHARED && all) {        // every slot of the chunk is seen by every row
        rows = a.bt.B * a.rows;
        sp.total = sp.len = (c + 1) * a.chunk;
    }
    if (row0 >= rows) return;
    __shared__ int s_bad[SHARED ? ROWS : 1];  // the tile's sequences that do not share the chunk
    if (SHARED && threadIdx.x < ROWS) s_bad[threadIdx.x] = 0;

    // ---- the wave's blocks: every W-th one of the chunk, but for those
    // between the sinks and every row's window
    const int per = a.chunk / kBlk, ac = chunk_of(sp, c);
    const int last = min((ac + 1) * per, (sp.total + kBlk - 1) / kBlk);
    const int gap0 = (a.sinks + kBlk - 1) / kBlk, gap1 = sp.lo / kBlk;
    auto settle = [&](int j) {  // j, or the next of the wave's blocks past the gap
        if (SHARED) return j;   // no window
        return j >= gap0 && j < gap1 ? j + (gap1 - j + W - 1) / W * W : j;
    };
    // The page of a block, by a scalar load (a vector load would be counted
    // behind the ring's transfers, and waiting for it would drain them): what
    // its entry holds, any entry past the last block.  It is looked at a block
    // later, so that nothing waits for the load.
    typedef const __attribute__((address_space(4))) int32_t *Entries;
    const Entries entries = (Entries)reinterpret_cast<uintptr_t>(a.kv.table + static_cast<int64_t>(sid) * a.kv.width);
    const int last_entry = max(min(((last - 1) >> a.kv.blk_shift) + 1, a.kv.width), 1) - 1;
    auto entry_of = [&](int j) { return entries[min(j >> a.kv.blk_shift, last_entry)]; };
    auto page_in = [&](int p) { return p >= 0 && p < a.kv.n_pages ? p : -1; };
    // a block without a page is read from page 0 and masked
    auto block_at = [&](int j, int page) {
        return kv_block(a.kv, a.layer, max(page, 0), head, j & ((1 << a.kv.blk_shift) - 1));
    };
    int j = settle(ac * per + wave);
    const bool any = j < last;
    int entry = entry_of(j);

    // ---- the ring: `slot` is the half read next and, once it is in
    // registers, the half that is refilled
    const uint32_t ring = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((SV_LDS uint8_t *)s_mem));
    const uint32_t mine = ring + wave * S::HALF, mine_scales = ring + S::SCALES_AT + wave * 256;
    uint32_t slot = 0;  // 0 .. N - 1
    int ji = j, jin = settle(j + W), pin = entry_of(jin);  // block to be requested, the one after it, its entry
    const uint8_t *bi = block_at(ji, page_in(entry));
    auto advance = [&]() {
        if (jin < last) {  // past the end the last block is requested again, so that the counts hold
            ji = jin;
            bi = block_at(ji, page_in(pin));
            jin = settle(jin + W);
            pin = entry_of(jin);
        }
    };
    // fp16, bf16: lane by lane what the lane will read; int8: as it lies
    const uint32_t k_from = ESZ == 2 ? (g * 32 + 8 * (col >> 2) + (col & 3)) * 16 : lane * 16;
    const uint32_t v_from = ESZ == 2 ? (g * D + col) * 16 : lane * 16;
    auto request_k = [&]() {
        half_to_lds<ONCE, 2048, (ESZ == 2 ? 64 : 1024), S::LOADS>(bi, fresh(k_from), mine + slot * (W * S::HALF));
        if constexpr (S::SCALES) {
            if (lane < 16) to_lds<ONCE>(bi + 64 * D + lane * 16, mine_scales + (slot >> 1) * (W * 256));
        }
    };
    auto request_v = [&]() {
        half_to_lds<ONCE, (ESZ == 2 ? 512 : 2048), (ESZ == 2 ? 256 : 1024), S::LOADS>(bi + S::HALF, fresh(v_from),
                                                                                     mine + slot * (W * S::HALF));
        advance();
    };
    auto turn = [&]() { slot = slot + 1 == S::N ? 0 : slot + 1; };
    const uint32_t staged = ring + S::STAGED, angles = ring + S::ANGLES;
    const int n_rows = min(ROWS, rows - row0);
    // rows numbered through the call's sequences where these share chunks
    const int at_b = SHARED ? 0 : b, at_row = SHARED ? b * a.rows + row0 : row0;
    stage_rows<D, W>(a, len, at_b, head, at_row, n_rows, wave, staged, angles);
    if (S::EARLY && any) {
        request_k();
        turn();
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::LOADS + S::SCALES) : "memory");  // all but the keys
    } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    // ---- queries, once every wave's pieces are there
    asm volatile("s_barrier" ::: "memory");
    if (a.rope.mode != SV_ROPE_NONE) {
        turn_rows<D, 64 * W>(a, len, at_b, at_row, n_rows, staged, angles);
        asm volatile("s_waitcnt lgkmcnt(0)\n s_barrier" ::: "memory");
    }
    typename Kd::KVec qf[RT][NC][Kd::kq];
    float rs[RT];
#pragma unroll
    for (int t = 0; t < RT; t++) rs[t] = take_queries<TYPE, D>(staged, 16 * t, n_rows, a.scale, qf[t]);
    asm volatile("s_barrier" ::: "memory");  // every wave has its queries
    if (any) {
#pragma unroll
        for (int i = 0; i < S::N / 2; i++) {
            if (i > 0 || !S::EARLY) {
                request_k();
                turn();
            }
            request_v();
            turn();
        }
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
    const int whole = sp.len + sp.n - a.window;  // with a window: from here on every row's window has begun
    // EVERY: all slots are seen by all rows.  A loop of its own where a kernel
    // has such chunks: what the other blocks' masks need would be kept in
    // registers across it.
    auto blocks = [&](auto every) __attribute__((always_inline)) {
    constexpr bool EVERY = decltype(every)::value;
    while (j < last) {
        const int s0 = j * kBlk;
        const int jn = settle(j + W), entry_n = EVERY ? 0 : entry_of(jn), page = EVERY ? 0 : page_in(entry);
        // ---- scores
        Raw<ESZ> kr[2 * NC], vr[ND];
        float ks[8], vs[8];  // int8: the scales of the lane group's eight slots
        if constexpr (ESZ == 2) {
            ring_read<S::LEAVE_K, 1024, 2 * NC>(mine + slot * (W * S::HALF) + lane * 16, kr);
        } else {
            ring_read<S::LEAVE_K, 1024, 32, 2 * NC>(
                mine + slot * (W * S::HALF) + (g * 32 + 8 * (col >> 2) + (col & 3)) * 8, kr);
            const uint32_t at = mine_scales + (slot >> 1) * (W * 256) + 32 * g;
            lds_read8(at, at + 16, ks);
            lds_read8(at + 128, at + 144, vs);
        }
        request_k();
        turn();
        float p[RT][8];
        {
            f4 acc[RT][2];
#pragma unroll
            for (int t = 0; t < RT; t++) acc[t][0] = acc[t][1] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int cc = 0; cc < NC; cc++) {
                const typename Kd::KVec k0 = widen<typename Kd::KVec>(kr[2 * cc]);
                const typename Kd::KVec k1 = widen<typename Kd::KVec>(kr[2 * cc + 1]);
#pragma unroll
                for (int n = Kd::kq - 1; n >= 0; n--)
#pragma unroll
                    for (int t = 0; t < RT; t++) {
                        acc[t][0] = mma(k0, qf[t][cc][n], acc[t][0]);
                        acc[t][1] = mma(k1, qf[t][cc][n], acc[t][1]);
                    }
            }
#pragma unroll
            for (int t = 0; t < RT; t++)
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    p[t][e] = acc[t][e >> 2][e & 3];
                    if constexpr (TYPE == SV_KV_I8) p[t][e] *= ks[e];
                }
        }

        // ---- what is visible, and the running softmax
        const bool edge = !EVERY && (page < 0 || s0 + kBlk > sp.len ||
                                     (!SHARED && a.window && s0 < whole && s0 + kBlk > a.sinks));
        // slots of the lane group that any row of the tile sees, and those that all see
        uint32_t any_sees = edge ? 0u : 0xFFu, all_see = 0xFFu;
        uint32_t seen[RT];  // slots of the lane group that the lane's row sees
#pragma unroll
        for (int t = 0; t < RT; t++) seen[t] = 0xFFu;
        if (edge) {
            // the rows' numbers are formed here, not kept in registers while
            // whole blocks go by
            const int at_lane = fresh(lane), to_g = at_lane >> 4, from = row0 + (at_lane & 15);
#pragma unroll
            for (int t = 0; t < RT; t++) {
                const int r = from + 16 * t;
                const bool live = r < rows;
                const int m = live ? a.by_group(r) : 0;
                const uint32_t mask = row_mask(a, b, m);
                const int pos = sp.len + __popc(mask & ((1u << m) - 1));
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int slot_e = s0 + 8 * to_g + e, nth = slot_e - sp.len;
                    bool sees = page >= 0 && slot_e < sp.total && (nth < 0 || (nth < sp.n && (mask >> nth & 1u)));
                    if (!SHARED && a.window && sees) {
                        int kpos = slot_e;
                        if (nth > 0 && a.bt.tree) kpos = sp.len + __popc(row_mask(a, b, nth) & ((1u << nth) - 1));
                        sees = pos - kpos < a.window || kpos < a.sinks;
                    }
                    if (!sees) {
                        p[t][e] = -INFINITY;
                        seen[t] &= ~(1u << e);
                    }
                    const uint32_t by = static_cast<uint32_t>(__ballot(live && sees) >> (16 * to_g)) & 0xFFFFu;
                    const uint32_t of = static_cast<uint32_t>(__ballot(live) >> (16 * to_g)) & 0xFFFFu;
                    if (by) any_sees |= 1u << e;
                    if (by != of) all_see &= ~(1u << e);
                }
            }
        }
        // int8: the weights carry the values' scales, so the maximum is that
        // of a weight with its scale
        float lift[8];
        if constexpr (TYPE == SV_KV_I8) {
#pragma unroll
            for (int e = 0; e < 8; e++) lift[e] = fmaxf(__builtin_amdgcn_logf(vs[e]), kLeastScale);
        }
        // The running maximum is taken up to a whole number: what it changes
        // by scales exactly, and seldom changes at all.
        float most[RT];
        bool far[RT];
#pragma unroll
        for (int t = 0; t < RT; t++) {
            auto with_scale = [&](int e) { return TYPE == SV_KV_I8 ? __builtin_fmaf(p[t][e], rs[t], lift[e]) : p[t][e]; };
            float top = with_scale(0);
#pragma unroll
            for (int e = 1; e < 8; e++) top = fmaxf(top, with_scale(e));
            top = row_max(top);
            most[t] = ceilf(TYPE == SV_KV_I8 ? top : top * rs[t]);
            far[t] = fabsf(most[t]) > kExact;
        }
        bool any_far = false;  // int8: a finite maximum too large for its scale
        if constexpr (TYPE == SV_KV_I8) {
#pragma unroll
            for (int t = 0; t < RT; t++) any_far |= far[t] && fabsf(most[t]) < INFINITY;
            any_far = __any(any_far);
            if (any_far) {
                // The scales are lost in such a sum: the maximum is that of
                // the scores, and the weights with their scales are taken in
                // fp32 below.
#pragma unroll
                for (int t = 0; t < RT; t++) {
                    float s = p[t][0];
#pragma unroll
                    for (int e = 1; e < 8; e++) s = fmaxf(s, p[t][e]);
                    s = row_max(s);
                    most[t] = far[t] ? ceilf(s * rs[t]) : most[t];
                }
            }
        }
#pragma unroll
        for (int t = 0; t < RT; t++) {
            // For fp16 products the maximum is held 15 too low, so that
            // weights go up to 2^15; not where fp32 would round that (by up
            // to 16, and 2^16 is past fp16): there scores are whole numbers
            // apart, and weights up to 1 keep what is known of them.
            if (TYPE != SV_KV_BF16 && !far[t]) most[t] -= 15.0f;
            const float now = fmaxf(mx[t], most[t]);
            const float base = now == -INFINITY ? 0.0f : now;
            const float keep = __builtin_amdgcn_exp2f(mx[t] - base);
            mx[t] = now;
            const float less = -base;
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                p[t][e] = __builtin_amdgcn_exp2f(TYPE == SV_KV_BF16 ? p[t][e] + less : __builtin_fmaf(p[t][e], rs[t], less));
                sum += p[t][e];
            }
            l[t] = l[t] * keep + sum;
            if (__any(keep != 1.0f)) {
#pragma unroll
                for (int i = 0; i < ND; i++) o[t][i] *= keep;
            }
            if constexpr (TYPE == SV_KV_I8) {
#pragma unroll
                for (int e = 0; e < 8; e++) p[t][e] *= vs[e];
                if (edge) {  // scales of hidden slots may be anything
#pragma unroll
                    for (int e = 0; e < 8; e++) p[t][e] = seen[t] >> e & 1u ? p[t][e] : 0.0f;
                }
            }
        }

        // ---- o += V^T P^T
        const uint8_t *blk = nullptr;
        if (!EVERY) blk = block_at(j, page);
        if constexpr (ESZ == 2) {
            ring_read<S::LEAVE_V, 1024, ND>(mine + slot * (W * S::HALF) + lane * 16, vr);
        } else {
            ring_read<S::LEAVE_V, 128, 0, ND>(mine + slot * (W * S::HALF) + (g * D + col) * 8, vr);
        }
        request_v();
        turn();
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
        if constexpr (TYPE == SV_KV_I8) {
            if (any_far) {
                if (EVERY) blk = block_at(j, page_in(entry_of(j)));
                // weights with scales that the maximum does not bound: in
                // fp32, slot by slot
                const int at_lane = fresh(lane), to_col = at_lane & 15, to_g = at_lane >> 4;
#pragma unroll 1
                for (int s = 0; s < kBlk; s++) {
                    float w[RT];
                    bool none = true;
#pragma unroll
                    for (int t = 0; t < RT; t++) {
                        w[t] = p[t][0];
#pragma unroll
                        for (int e = 1; e < 8; e++) w[t] = (s & 7) == e ? p[t][e] : w[t];
                        w[t] = far[t] ? w[t] : 0.0f;
                        w[t] = __uint_as_float(__builtin_amdgcn_ds_bpermute(4 * (16 * (s >> 3) + to_col), __float_as_uint(w[t])));
                        none &= w[t] == 0.0f;
                    }
                    if (__all(none)) continue;
                    const uint8_t *v = blk + 32 * D + ((s >> 3) * D + 4 * to_g) * 8 + (s & 7);
#pragma unroll
                    for (int i = 0; i < ND; i++) {
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const float y = static_cast<float>(static_cast<int8_t>(gld(v + (16 * i + k) * 8)));
#pragma unroll
                            for (int t = 0; t < RT; t++) o[t][i][k] += w[t] * y;
                        }
                        asm volatile("" ::: "memory");  // a few loads at a time, for the registers' sake
                    }
                }
#pragma unroll
                for (int t = 0; t < RT; t++)
#pragma unroll
                    for (int e = 0; e < 8; e++) p[t][e] = far[t] ? 0.0f : p[t][e];
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
                const int at_lane = fresh(lane), to_col = at_lane & 15, to_g = at_lane >> 4;
#pragma unroll 1
                for (int s = 0; s < kBlk; s++) {
                    const uint8_t *v = blk + (32 * D + ((s >> 3) * D + 4 * to_g) * 8 + (s & 7)) * ESZ;
#pragma unroll
                    for (int t = 0; t < RT; t++) {
                        float w = p[t][0];
#pragma unroll
                        for (int e = 1; e < 8; e++) w = (s & 7) == e ? p[t][e] : w;
                        const int from = 16 * (s >> 3) + to_col;
                        w = __uint_as_float(__builtin_amdgcn_ds_bpermute(4 * from, __float_as_uint(w)));
                        const bool sees = __builtin_amdgcn_ds_bpermute(4 * from, seen[t]) >> (s & 7) & 1;
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
        j = jn;
        entry = entry_n;
    }
    };
    if constexpr (SHARED) {
        if (all) blocks(std::true_type{});
        else blocks(std::false_type{});
    } else {
        blocks(std::false_type{});
    }
    // the last requests land before the ring's memory is used again
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // ---- the waves' results joined, wave by wave
    float *s_o = reinterpret_cast<float *>(s_mem);  // [W][ROWS][LD]
    __syncthreads();
#pragma unroll
    for (int t = 0; t < RT; t++) {
        l[t] = row_sum(l[t]);
        if (g == 0) {
            s_m[wave][16 * t + col] = mx[t];
            s_l[wave][16 * t + col] = l[t];
        }
#pragma unroll
        for (int i = 0; i < ND; i++)
            *reinterpret_cast<f4 *>(s_o + (wave * ROWS + 16 * t + col) * LD + 16 * i + 4 * g) = o[t][i];
    }
    if constexpr (SHARED) {
        if (all) find_strangers(a, sid, named, c, row0, n_rows, 64 * W, s_bad);
    }
    __syncthreads();
    const int n = min(ROWS, rows - row0);
    const int64_t part0 = ((static_cast<int64_t>(b) * heads + head) * a.chunks + c) * a.rows + row0;
    for (int i = threadIdx.x; i < n * (D / 4); i += 64 * W) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        int64_t part = part0;
        bool bad = false;
        if constexpr (SHARED) {
            if (all) {
                const int of = a.by_rows(row0 + r), own = row0 + r - of * a.rows;
                bad = s_bad[of - a.by_rows(row0)];
                part = ((static_cast<int64_t>(of) * heads + head) * a.chunks + c) * a.rows + own - r;
                if (own >= kv_rows_of(a.bt.n_new, of, a.bt.M) * a.group) continue;
            }
        }
        float top = s_m[0][r];
#pragma unroll
        for (int w = 1; w < W; w++) top = fmaxf(top, s_m[w][r]);
        float sum = 0.0f;
        f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < W; w++) {
            const float by = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s_m[w][r] - top);
            sum += s_l[w][r] * by;
            v += by * *reinterpret_cast<const f4 *>(s_o + (w * ROWS + r) * LD + d);
        }
        if (alone) {
            const bool over = a.max_len && sp.len + sp.n > a.max_len;
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
            // its own place in the first wave's sums, which no other thread reads
            *reinterpret_cast<f4 *>(s_o + r * LD + d) = over ? f4{NAN, NAN, NAN, NAN} : v * inv;
            if (over && i == 0) kv_flag(a.kv, SV_KV_OVER_MAX);
        } else {
            *(SV_GLOBAL f4 *)(a.part_o + (part + r) * D + d) = v;
            if (d == 0) {
                gst(a.part_m + part + r, bad ? NAN : top);
                gst(a.part_l + part + r, sum);
            }
        }
    }
    if (alone) {
        __syncthreads();
        finish_rows(a, s_o, LD, b, head, row0, n);
    }
}

// Launches a variant: a workgroup per chunk that there can be, and row group.
template <int TYPE, int D, int RT, typename Args>
static int launch_one(const Args &a, int64_t units, hipStream_t st) {
    using S = Shape<TYPE, D, RT>;
    static_assert(S::LDS <= kMaxLds, "LDS");
    if constexpr (S::LDS > 65536) {  // above the default, allowed once for each device
        static std::atomic<uint64_t> allowed{0};
        int dev = 0;
        int rc = hip_check(hipGetDevice(&dev), "kv_attention: device");
        if (rc) return rc;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (!(allowed.load() & bit)) {
            rc = hip_check(hipFuncSetAttribute(reinterpret_cast<const void *>(&kv_attn_kernel<TYPE, D, RT, Args>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS),
                           "kv_attention: LDS size");
            if (rc) return rc;
            allowed.fetch_or(bit);
        }
    }
    unsigned grid = static_cast<unsigned>((units + 7) / 8 * 8 * a.tiles);
    if constexpr (__is_same(Args, AttnShared)) grid += a.shared_grid;
    hipLaunchKernelGGL((kv_attn_kernel<TYPE, D, RT, Args>), dim3(grid), dim3(64 * S::W), S::LDS, st, a);
    return hip_check(hipGetLastError(), "kv_attention launch");
}

template <int TYPE, int D, typename Args>
static int launch_dim(const Args &a, int rt, int64_t units, hipStream_t st) {
    if constexpr (D <= 64) {
        if (rt == 4) return launch_one<TYPE, D, 4, Args>(a, units, st);
    }
    if constexpr (D <= 128) {
        if (rt == 2) return launch_one<TYPE, D, 2, Args>(a, units, st);
    }
    return launch_one<TYPE, D, 1, Args>(a, units, st);
}

template <int TYPE, typename Args>
static int launch_type(const Args &a, int rt, int64_t units, hipStream_t st) {
    switch (a.kv.dim) {
        case 32: return launch_dim<TYPE, 32, Args>(a, rt, units, st);
        case 64: return launch_dim<TYPE, 64, Args>(a, rt, units, st);
        case 96: return launch_dim<TYPE, 96, Args>(a, rt, units, st);
        case 128: return launch_dim<TYPE, 128, Args>(a, rt, units, st);
        case 160: return launch_dim<TYPE, 160, Args>(a, rt, units, st);
        case 192: return launch_dim<TYPE, 192, Args>(a, rt, units, st);
        case 224: return launch_dim<TYPE, 224, Args>(a, rt, units, st);
        case 256: return launch_dim<TYPE, 256, Args>(a, rt, units, st);
    }
    return fail(SV_ERR_SHAPE, "kv_attention: unsupported head dimension");
}

#if SV_INST_KV == 1
int attn_launch_f16(const AttnArgs &a, int rt, int64_t units, hipStream_t st) { return launch_type<SV_KV_F16>(a, rt, units, st); }
int attn_launch_f16(const AttnShared &a, int rt, int64_t units, hipStream_t st) { return launch_type<SV_KV_F16>(a, rt, units, st); }
#elif SV_INST_KV == 30
int attn_launch_bf16(const AttnArgs &a, int rt, int64_t units, hipStream_t st) { return launch_type<SV_KV_BF16>(a, rt, units, st); }
int attn_launch_bf16(const AttnShared &a, int rt, int64_t units, hipStream_t st) { return launch_type<SV_KV_BF16>(a, rt, units, st); }
#else
int attn_launch_i8(const AttnArgs &a, int rt, int64_t units, hipStream_t st) { return launch_type<SV_KV_I8>(a, rt, units, st); }
int attn_launch_i8(const AttnShared &a, int rt, int64_t units, hipStream_t st) { return launch_type<SV_KV_I8>(a, rt, units, st); }
#endif

}  // namespace sv
