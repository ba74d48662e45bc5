// kv_attn.hip - host side of the cache's attention, and the join of the
// chunks' partial softmaxes.
#include <algorithm>

#include "kv_attn.h"

namespace sv {

// The join of a row's chunks c: with M = max m_c,
//   out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c,
// one workgroup a row; its threads take four elements each of the head
// dimension and one of `parts` shares of the chunks (chunk number modulo
// parts, each share in chunk order, then the shares in order), so the sums
// do not depend on how many chunks a launch provides for.
constexpr int kJoin = 256, kJoinTile = 1024;
__global__ __launch_bounds__(kJoin) void kv_attn_join_kernel(AttnArgs a) {
    fetch_args<sizeof(AttnArgs)>();
    __shared__ float s_w[kJoinTile], s_wl[kJoinTile];
    __shared__ __align__(16) float s_v[kJoin * 4];
    __shared__ float s_l[kJoin / 8], s_top[kJoin / 64];
    typedef float f4 __attribute__((ext_vector_type(4)));
    const int r = blockIdx.x, head = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int sid = a.bt.seq ? gld(a.bt.seq + b) : b;
    if (sid < 0 || sid >= a.kv.seqs) return;
    const Span sp = span_of(a, static_cast<int>(kv_len_of(a.kv, sid)), kv_rows_of(a.bt.n_new, b, a.bt.M));
    if (r >= sp.n * a.group) return;
    const int D = a.kv.dim, quads = D / 4, parts = kJoin / quads;
    const int n = chunks_of(a, sp);
    const int64_t base = (static_cast<int64_t>(b) * a.kv.heads + head) * a.chunks * a.rows + r;
    float top = -INFINITY;
    for (int c = tid; c < n; c += kJoin) top = fmaxf(top, gld(a.part_m + base + static_cast<int64_t>(c) * a.rows));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if ((tid & 63) == 0) s_top[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
    const int part = tid / quads, d = tid % quads * 4;
    f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
    for (int at = 0; at < n && top != -INFINITY; at += kJoinTile) {
        const int upto = min(n - at, kJoinTile);
        for (int i = tid; i < upto; i += kJoin) {
            const int64_t c = base + static_cast<int64_t>(at + i) * a.rows;
            const float w = __builtin_amdgcn_exp2f(gld(a.part_m + c) - top);
            s_w[i] = w;
            s_wl[i] = w * gld(a.part_l + c);
        }
        __syncthreads();
        if (part < parts) {
            // the chunks of the sinks and those after them: two runs of
            // consecutive chunk numbers
            for (int run = 0; run < 2; run++) {
                const int lo = max(at, run ? sp.first : 0), hi = min(at + upto, run ? n : sp.first);
                const int shift = run ? sp.jump - sp.first : 0;
                int c = lo + ((part - (lo + shift)) % parts + parts) % parts;
#pragma unroll 4
                for (; c < hi; c += parts) {
                    v += s_w[c - at] * *(const SV_GLOBAL f4 *)(a.part_o + (base + static_cast<int64_t>(c) * a.rows) * D + d);
                    l += s_wl[c - at];
                }
            }
        }
        __syncthreads();
    }
    if (part < parts) {
        *reinterpret_cast<f4 *>(s_v + part * D + d) = v;
        if (d == 0) s_l[part] = l;
    }
    __syncthreads();
    float x = 0.0f;
    if (tid < D) {
        float sum = s_l[0];
        x = s_v[tid];
        for (int i = 1; i < parts; i++) {
            x += s_v[i * D + tid];
            sum += s_l[i];
        }
        const bool over = a.max_len && sp.len + sp.n > a.max_len;
        if (over && tid == 0) kv_flag(a.kv, SV_KV_OVER_MAX);
        x = over ? NAN : x * (sum != 0.0f ? 1.0f / sum : 0.0f);
    }
    __syncthreads();
    if (tid < D) s_v[tid] = x;
    __syncthreads();
    finish_rows(a, s_v, D, b, head, r, 1);
}

// Chunks that a sequence can have: of its whole length, or of what a window
// and the sinks can touch.
static int64_t chunks_within(int64_t bound, int64_t window, int64_t sinks, int64_t chunk) {
    const int64_t all = (bound + chunk - 1) / chunk;
    if (!window) return all;
    const int64_t most = (sinks + chunk - 1) / chunk + (window + SV_MAX_M + chunk - 1) / chunk + 1;
    return std::min(all, most);
}

// Slots of a chunk when the caller leaves the choice: the shortest with which
// the launch is one round of workgroups (256 compute units hold one wide or
// two narrow workgroups each).  Without a window the sequences of a batch are
// seldom all as long as the longest: half a round more is allowed for.  Past
// one round of 2048 the length evens out the last round.  Measured in us, 128
// heads of 8 and a group of 5:
//   5 x 4099 slots, 8 heads, fp16          256: 22, 384: 25, 640: 37
//   8 rows, window 1024, 8 heads of 96     384: 24, 512: 20, 640: 24
//   4 trees of up to 8191, 8 heads of 64   256: 50, 384: 36, 512: 43
//   16 sequences up to 16384, int8         1024: 94, 1536: 90, 2048: 98
//   32 sequences, window 4096, fp16        1024: 152, 1536: 148, 2048: 166
// A sequence that fits one short chunk needs no join (300 slots: 11 against
// 14 with chunks of 256).
static int chunk_rule(int64_t B, int64_t heads, int dim, int64_t bound, int64_t window, int64_t sinks) {
    if (bound <= 512) return static_cast<int>((bound + 127) / 128 * 128);
    for (int c = 256; c <= 2048; c += 128) {
        int64_t room = attn_wide(dim, c) ? 256 : 512;
        if (B > 1 && !window) room += room / 2;
        const int64_t pairs = B * heads;
        // of a window that lies anywhere: window / c + 1 chunks on average
        const int64_t units = window && window + sinks < bound ? pairs * ((sinks + c - 1) / c + 1) + pairs * window / c
                                                               : pairs * ((bound + c - 1) / c);
        if (units <= room) return c;
    }
    return 1536;
}

struct Plan {
    int64_t bound, units;
    int rt;
    size_t o_m, o_l, bytes;
};

static int plan_of(const KvDev &d, const sv_kv_batch *bt, const sv_kv_attn *at, AttnArgs *a, Plan *p) {
    SV_REQUIRE(at, SV_ERR_ARG, "kv_attention: NULL arguments");
    SV_REQUIRE(at->q_heads >= 1 && at->q_heads % d.heads == 0 && at->q_heads / d.heads <= 64, SV_ERR_SHAPE,
               "kv_attention: q_heads must be a multiple of heads, at most 64 times");
    SV_REQUIRE(at->scale > 0.0f && at->scale <= 3.0e38f, SV_ERR_ARG, "kv_attention: scale must be positive and finite");
    SV_REQUIRE(at->window >= 0 && at->sinks >= 0 && at->sinks < (1 << 30), SV_ERR_ARG,
               "kv_attention: window and sinks must not be negative, sinks below 2^30");
    SV_REQUIRE(at->window > 0 || at->sinks == 0, SV_ERR_ARG, "kv_attention: sinks need a window");
    SV_REQUIRE(at->max_len >= 0, SV_ERR_ARG, "kv_attention: max_len must not be negative");
    SV_REQUIRE(at->chunk >= 0 && at->chunk % 128 == 0 && at->chunk <= (1 << 24), SV_ERR_ARG,
               "kv_attention: chunk must be a multiple of 128, at most 2^24");
    const int rc = kv_check_rope(d, at->rope, "kv_attention");
    if (rc) return rc;
    const int64_t cap = static_cast<int64_t>(d.width) * d.page;
    p->bound = at->max_len && at->max_len < cap ? at->max_len : cap;
    a->kv = d;
    a->bt = *bt;
    a->rope = at->rope ? *at->rope : sv_kv_rope{};
    a->q_heads = at->q_heads;
    a->group = at->q_heads / d.heads;
    a->rows = bt->M * a->group;
    a->window = at->window;
    a->sinks = at->sinks;
    a->max_len = at->max_len;
    a->chunk = at->chunk ? at->chunk : chunk_rule(bt->B, d.heads, d.dim, p->bound, at->window, at->sinks);
    const int64_t chunks = chunks_within(p->bound, at->window, at->sinks, a->chunk);
    a->chunks = static_cast<int32_t>(chunks);
    a->wide = attn_wide(d.dim, a->chunk);
    a->scale = at->scale * 1.44269504088896340736f;
    p->rt = attn_tiles_per_wave(d.dim, a->rows);
    a->tiles = (a->rows + 16 * p->rt - 1) / (16 * p->rt);
    a->by_group = div_by(a->group);
    a->by_chunk = div_by(a->chunk);
    a->by_tiles = div_by(a->tiles);
    a->by_heads = div_by(d.heads);
    a->by_turns = div_by(std::max(1, a->rope.rot / 8));
    p->units = static_cast<int64_t>(bt->B) * d.heads * chunks;
    SV_REQUIRE(p->units * a->tiles < (1ll << 24), SV_ERR_SHAPE, "kv_attention: too many chunks (use a longer chunk)");
    p->bytes = p->o_m = p->o_l = 0;
    if (chunks > 1) {
        const size_t parts = static_cast<size_t>(bt->B) * d.heads * chunks * a->rows;
        p->o_m = (parts * d.dim * 4 + 255) / 256 * 256;
        p->o_l = p->o_m + (parts * 4 + 255) / 256 * 256;
        p->bytes = p->o_l + (parts * 4 + 255) / 256 * 256;
    }
    return SV_OK;
}

}  // namespace sv

using namespace sv;

extern "C" size_t sv_kv_attention_workspace_bytes(const sv_kv *kv, const sv_kv_batch *batch, const sv_kv_attn *attn) {
    KvDev d;
    AttnArgs a{};
    Plan p;
    if (kv_check(kv, "kv_attention", &d) || kv_check_batch(d, batch, "kv_attention", SV_MAX_M) ||
        plan_of(d, batch, attn, &a, &p))
        return 0;
    return p.bytes;
}

extern "C" int sv_kv_attention(const sv_kv *kv, int32_t layer, const sv_kv_batch *batch, const sv_kv_attn *attn,
                               const float *q, float *out, const sv_epilogue *ep, void *workspace, size_t ws_bytes,
                               void *stream) {
    KvDev d;
    AttnArgs a{};
    Plan p;
    int rc = kv_check(kv, "kv_attention", &d);
    if (!rc) rc = kv_check_batch(d, batch, "kv_attention", SV_MAX_M);
    if (!rc) rc = plan_of(d, batch, attn, &a, &p);
    if (rc) return rc;
    SV_REQUIRE(layer >= 0 && layer < d.layers, SV_ERR_ARG, "kv_attention: layer out of range");
    const bool quant = ep && ep->mode != SV_EP_NONE;
    SV_REQUIRE(q && (out || quant), SV_ERR_ARG, "kv_attention: NULL buffer");
    SV_REQUIRE(aligned(q, 16) && (!out || aligned(out, 16)), SV_ERR_ALIGN,
               "kv_attention: q and out must be 16-byte aligned");
    if (quant) {
        SV_REQUIRE(ep->mode == SV_EP_QUANT && ep->src == 0, SV_ERR_ARG,
                   "kv_attention: the epilogue's mode must be SV_EP_QUANT and its src 0");
        SV_REQUIRE(ep->q && ep->d && ep->s16 && ep->sumsq, SV_ERR_ARG, "kv_attention: NULL epilogue buffer");
        SV_REQUIRE((!ep->gamma || aligned(ep->gamma, 4)) && aligned(ep->d, 4) && aligned(ep->s16, 4) &&
                       aligned(ep->sumsq, 4),
                   SV_ERR_ALIGN, "kv_attention: fp32/int32 buffers must be 4-byte aligned");
        a.ep = *ep;
    }
    SV_REQUIRE(p.bytes == 0 || (workspace && ws_bytes >= p.bytes), SV_ERR_WORKSPACE,
               "kv_attention: workspace needs " + std::to_string(p.bytes) + " bytes");
    SV_REQUIRE(p.bytes == 0 || aligned(workspace, 256), SV_ERR_ALIGN,
               "kv_attention: the workspace must be 256-byte aligned");
    a.q = q;
    a.out = out;
    a.layer = layer;
    if (p.bytes) {
        uint8_t *ws = static_cast<uint8_t *>(workspace);
        a.part_o = reinterpret_cast<float *>(ws);
        a.part_m = reinterpret_cast<float *>(ws + p.o_m);
        a.part_l = reinterpret_cast<float *>(ws + p.o_l);
    }
    hipStream_t st = as_stream(stream);
    rc = d.type == SV_KV_F16    ? attn_launch_f16(a, p.rt, p.units, st)
         : d.type == SV_KV_BF16 ? attn_launch_bf16(a, p.rt, p.units, st)
                                : attn_launch_i8(a, p.rt, p.units, st);
    if (rc || a.chunks == 1) return rc;
    hipLaunchKernelGGL(kv_attn_join_kernel, dim3(a.rows, d.heads, batch->B), dim3(kJoin), 0, st, a);
    return hip_check(hipGetLastError(), "kv_attention join launch");
}
