// kv_attn.h - argument block of the cache's attention kernels and the
// launchers of their variants (one source compiled per cache type).
#pragma once

#include "kv_internal.h"

namespace sv {

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
};

// What a sequence's rows see, in whole chunks.
struct Span {
    int64_t len;       // committed slots
    int64_t total;     // slots that can be seen: committed and new, within the table row
    int64_t lo;        // first slot inside the first row's window
    int n;             // rows
    int first;         // chunks [0, first) hold the sinks; the next one of the launch is chunk `jump`
    int jump;
    int end;           // one past the last chunk
};

__device__ __forceinline__ Span span_of(const AttnArgs &a, int b, int sid) {
    Span s;
    s.len = kv_len_of(a.kv, sid);
    s.n = kv_rows_of(a.bt.n_new, b, a.bt.M);
    const int64_t cap = static_cast<int64_t>(a.kv.width) * a.kv.page;
    s.total = s.len + s.n < cap ? s.len + s.n : cap;
    s.lo = a.window && s.len >= a.window ? s.len - a.window + 1 : 0;
    s.end = static_cast<int>((s.total + a.chunk - 1) / a.chunk);
    s.first = 0;
    s.jump = 0;
    if (s.lo > a.sinks) {
        s.first = (a.sinks + a.chunk - 1) / a.chunk;
        s.jump = static_cast<int>(s.lo / a.chunk);
        if (s.jump < s.first) s.jump = s.first;
    }
    return s;
}
// Chunk of a launch's index c; at or past s.end: none.
__device__ __forceinline__ int chunk_of(const Span &s, int c) { return c < s.first ? c : s.jump + (c - s.first); }

__device__ __forceinline__ uint32_t row_mask(const AttnArgs &a, int b, int m) {
    return a.bt.tree ? gld(a.bt.tree + static_cast<int64_t>(b) * a.bt.M + m) : (2u << m) - 1;
}
// Writes the finished values of rows row0 .. row0 + n - 1 of a head from LDS:
// out, and the next projection's input as sv_quantize_act_q8 makes it of out
// (a half wave per 32 values, the same reductions in the same order).
__device__ __forceinline__ void finish_rows(const AttnArgs &a, const float *vals, int ld, int b, int head, int row0,
                                            int n) {
    const int nb = a.kv.dim / 32, lane = threadIdx.x & 31;
    for (int it = threadIdx.x >> 5; it < n * nb; it += blockDim.x >> 5) {
        const int i = it / nb, blk = it % nb, r = row0 + i;
        const int hq = head * a.group + r % a.group;
        const int64_t row = (static_cast<int64_t>(b) * a.bt.M + r / a.group) * a.q_heads + hq;
        const float x = vals[i * ld + 32 * blk + lane];
        const int64_t e = row * a.kv.dim + 32 * blk + lane;
        if (a.out) gst(a.out + e, x);
        if (a.ep.mode == SV_EP_NONE) continue;
        const float y = a.ep.gamma ? x * gld(a.ep.gamma + hq * a.kv.dim + 32 * blk + lane) : x;
        float m = fabsf(y);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 32));
        const float d = m / 127.0f, id = d != 0.0f ? 1.0f / d : 0.0f;
        const int q = static_cast<int>(fminf(fmaxf(roundf(y * id), -127.0f), 127.0f));
        int s = q;
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) s += __shfl_xor(s, o, 32);
        float sq = x * x;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sq += __shfl_xor(sq, o, 32);
        gst(a.ep.q + e, static_cast<int8_t>(q));
        if ((lane & 15) == 0) gst(a.ep.s16 + e / 16, s);
        if (lane == 0) {
            gst(a.ep.d + e / 32, d);
            gst(a.ep.sumsq + e / 32, sq);
        }
    }
}

// Row tiles of 16 that one wave holds, by the rows of a head.
inline int attn_tiles_per_wave(int dim, int rows) { return dim > 128 || rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

int attn_launch_f16(const AttnArgs &a, int rt, dim3 grid, hipStream_t st);
int attn_launch_bf16(const AttnArgs &a, int rt, dim3 grid, hipStream_t st);
int attn_launch_i8(const AttnArgs &a, int rt, dim3 grid, hipStream_t st);

}  // namespace sv
