// kv_attn.h - argument block of the cache's attention kernels and the
// launchers of their variants (one source compiled per cache type).
#pragma once

#include "kv_internal.h"

namespace sv {

// Division of 0 <= x < 2^31 by a number that the host knows.
struct Div {
    uint32_t m, sh;
    __device__ __forceinline__ int operator()(int x) const {
        return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(x)) * m >> sh);
    }
};
inline Div div_by(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) l++;
    return Div{static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

struct AttnArgs {
    KvDev kv;
    sv_kv_batch bt;
    sv_kv_rope rope;
    sv_epilogue ep;
    const float *q;
    float *out;
    // partial softmaxes of the chunks: [B][heads][chunks][rows] each, the
    // weighted sums [dim] floats a row; rows = M * group
    float *part_o, *part_m, *part_l;
    int32_t layer, q_heads, group, rows;
    int32_t window, sinks;
    int32_t max_len;   // 0 = not checked
    int32_t chunk;     // slots
    int32_t chunks;    // of a launch: as many as any sequence can have
    int32_t tiles;     // workgroups that share a (sequence, head, chunk): row groups
    float scale;       // times log2(e)
    Div by_group, by_chunk, by_tiles, by_heads, by_turns;  // by_turns: by rot / 8
};

// What a sequence's rows see, in whole chunks.  Slots fit 32 bits (width *
// page is below 2^31 - 65536).
struct Span {
    int len;      // committed slots
    int total;    // slots that can be seen: committed and new, within the table row
    int lo;       // first slot inside the first row's window
    int n;        // rows
    int first;    // chunks [0, first) hold the sinks; the next one of the launch is chunk `jump`
    int jump;
    int end;      // one past the last chunk
};

__device__ __forceinline__ Span span_of(const AttnArgs &a, int len, int n) {
    Span s;
    s.len = len;
    s.n = n;
    const int cap = a.kv.width * a.kv.page;
    s.total = s.len + s.n < cap ? s.len + s.n : cap;
    s.lo = a.window && s.len >= a.window ? s.len - a.window + 1 : 0;
    s.end = s.total ? a.by_chunk(s.total - 1) + 1 : 0;  // total + chunk may pass 2^31
    s.first = 0;
    s.jump = 0;
    if (s.lo > a.sinks) {
        s.first = a.by_chunk(a.sinks + a.chunk - 1);
        s.jump = a.by_chunk(s.lo);
        if (s.jump < s.first) s.jump = s.first;
    }
    return s;
}
// Chunks of a sequence in a launch.
__device__ __forceinline__ int chunks_of(const AttnArgs &a, const Span &s) {
    return min(a.chunks, s.first + max(s.end - s.jump, 0));
}
// Chunk of a launch's index c; at or past s.end: none.
__device__ __forceinline__ int chunk_of(const Span &s, int c) { return c < s.first ? c : s.jump + (c - s.first); }

// A value that the compiler takes as new, so that what follows from it is
// formed where it is used and not kept in registers across a loop.
__device__ __forceinline__ int fresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ uint32_t row_mask(const AttnArgs &a, int b, int m) {
    return a.bt.tree ? gld(a.bt.tree + static_cast<int64_t>(b) * a.bt.M + m) : (2u << m) - 1;
}
// Sums and maxima over lanes by moves that need no index register (an index
// would be kept across the kernel's loops).  Over 32 lanes: lanes 16 apart,
// then rotations within 16 lanes by 8, 4, 2 and 1: with the halves equal,
// each is the exchange of lanes that far apart.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ int dpp_i32(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
constexpr int kRor = 0x120;  // row_ror
__device__ __forceinline__ void swap16(float v, float *a, float *b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    *a = __uint_as_float(r[0]);
    *b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap32(float v, float *a, float *b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    *a = __uint_as_float(r[0]);
    *b = __uint_as_float(r[1]);
}
__device__ __forceinline__ float max32(float v) {
    float a, b;
    swap16(v, &a, &b);
    v = fmaxf(a, b);
    v = fmaxf(v, dpp_f32<kRor + 8>(v));
    v = fmaxf(v, dpp_f32<kRor + 4>(v));
    v = fmaxf(v, dpp_f32<kRor + 2>(v));
    return fmaxf(v, dpp_f32<kRor + 1>(v));
}
__device__ __forceinline__ float sum32(float v) {
    float a, b;
    swap16(v, &a, &b);
    v = a + b;
    v += dpp_f32<kRor + 8>(v);
    v += dpp_f32<kRor + 4>(v);
    v += dpp_f32<kRor + 2>(v);
    return v + dpp_f32<kRor + 1>(v);
}
__device__ __forceinline__ int sum16(int v) {
    v += dpp_i32<kRor + 8>(v);
    v += dpp_i32<kRor + 4>(v);
    v += dpp_i32<kRor + 2>(v);
    return v + dpp_i32<kRor + 1>(v);
}
// Sum of the lanes up to and with this one.
__device__ __forceinline__ int scan64(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15, 31
    return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
}

// Writes the finished values of rows row0 .. row0 + n - 1 of a head from LDS:
// out, and the next projection's input as sv_quantize_act_q8 makes it of out
// (a half wave per 32 values, the same reductions in the same order).
__device__ __forceinline__ void finish_rows(const AttnArgs &a, const float *vals, int ld, int b, int head, int row0,
                                            int n) {
    const int tid = fresh(threadIdx.x);
    const int nb = a.kv.dim / 32, lane = tid & 31;
    for (int it = tid >> 5; it < n * nb; it += blockDim.x >> 5) {
        const int i = it / nb, blk = it % nb, r = row0 + i;
        const int m = a.by_group(r), hq = head * a.group + r - m * a.group;
        const int64_t row = (static_cast<int64_t>(b) * a.bt.M + m) * a.q_heads + hq;
        const float x = vals[i * ld + 32 * blk + lane];
        const int64_t e = row * a.kv.dim + 32 * blk + lane;
        if (a.out) gst(a.out + e, x);
        if (a.ep.mode == SV_EP_NONE) continue;
        const float y = a.ep.gamma ? x * gld(a.ep.gamma + hq * a.kv.dim + 32 * blk + lane) : x;
        const float d = max32(fabsf(y)) / 127.0f, id = d != 0.0f ? 1.0f / d : 0.0f;
        const int q = static_cast<int>(fminf(fmaxf(roundf(y * id), -127.0f), 127.0f));
        const int s = sum16(q);
        const float sq = sum32(x * x);
        gst(a.ep.q + e, static_cast<int8_t>(q));
        if ((lane & 15) == 0) gst(a.ep.s16 + e / 16, s);
        if (lane == 0) {
            gst(a.ep.d + e / 32, d);
            gst(a.ep.sumsq + e / 32, sq);
        }
    }
}

constexpr int kMaxLds = 79 * 1024;  // two workgroups a compute unit

// Row tiles of 16 that one wave holds: all rows of a head where the registers
// allow it, so that a block is read and widened once for them (us: 64 rows of
// 64 in four tiles 25 against 32 in two twice; 25 rows of 128 in two tiles,
// 131001 slots, 95 against 148 in one twice, int8 batch 79 against 93).
inline int attn_tiles_per_wave(int dim, int rows) { return dim > 128 || rows <= 16 ? 1 : rows <= 32 || dim > 64 ? 2 : 4; }

int attn_launch_f16(const AttnArgs &a, int rt, int64_t units, hipStream_t st);
int attn_launch_bf16(const AttnArgs &a, int rt, int64_t units, hipStream_t st);
int attn_launch_i8(const AttnArgs &a, int rt, int64_t units, hipStream_t st);

}  // namespace sv
