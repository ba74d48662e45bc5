// kv_attn.hip - host side of the cache's attention, and the join of the
// chunks' partial softmaxes.
#include <algorithm>

#include "kv_attn.h"

namespace sv {

// The join of a row's chunks c: with M = max m_c,
//   out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c
// in kShares shares (chunk number modulo kShares), each in chunk order, then
// the shares in order: the sums depend neither on how many chunks a launch
// provides for nor on the kernel that forms them.
//
// Both kernels are bound by latency: the sequence, its length, the maxima and
// the sums are loads that wait for one another, so what is likely to be used
// is requested before the length is known.
constexpr int kShares = 8, kJoin = 256;
typedef float f4 __attribute__((ext_vector_type(4)));

struct Parts {
    const float *o, *m, *l;  // of the row's first chunk
    int64_t step;            // rows between chunks
    int D;
    __device__ Parts(const AttnArgs &a, int b, int head, int r) {
        const int64_t base = (static_cast<int64_t>(b) * a.kv.heads + head) * a.chunks * a.rows + r;
        step = a.rows;
        D = a.kv.dim;
        o = a.part_o + base * D;
        m = a.part_m + base;
        l = a.part_l + base;
    }
    __device__ float m_at(int c) const { return gld(m + c * step); }
    __device__ float l_at(int c) const { return gld(l + c * step); }
    __device__ f4 o_at(int c, int d) const { return *(const SV_GLOBAL f4 *)(o + c * step * D + d); }
};
// The launch's chunks are two runs of consecutive chunk numbers: [0, first)
// as they are, the others `jump - first` ahead of their index.
struct Run {
    int from, to, shift;
    __device__ Run(const Span &sp, int n, int nth)
        : from(nth ? sp.first : 0), to(nth ? n : min(n, sp.first)), shift(nth ? sp.jump - sp.first : 0) {}
};
__device__ __forceinline__ void flag_over(const AttnArgs &a, const Span &sp) {
    if (a.max_len && sp.len + sp.n > a.max_len) kv_flag(a.kv, SV_KV_OVER_MAX);
}
__device__ __forceinline__ f4 joined(const AttnArgs &a, const Span &sp, f4 x, float sum) {
    if (a.max_len && sp.len + sp.n > a.max_len) return f4{NAN, NAN, NAN, NAN};
    return x * (sum != 0.0f ? 1.0f / sum : 0.0f);
}

// Few rows: one workgroup each, a share to every dim / 4 threads.
constexpr int kWeights = 1024, kAhead = 8;
__global__ __launch_bounds__(512) void kv_attn_join_kernel(AttnArgs a) {
    __shared__ float s_w[kWeights], s_wl[kWeights];
    __shared__ __align__(16) float s_v[kShares * kMaxDim];
    __shared__ float s_l[kShares], s_top[8];
    fetch_args<sizeof(AttnArgs)>();
    const int r = blockIdx.x, head = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, threads = blockDim.x;
    const int D = a.kv.dim, quads = D / 4;
    const Parts at(a, b, head, r);
    const int group = tid / quads, d = (tid - group * quads) * 4;
    float m_ahead = 0.0f, l_ahead = 0.0f;
    f4 ahead[kAhead];
    if (tid < a.chunks) {
        m_ahead = at.m_at(tid);
        l_ahead = at.l_at(tid);
    }
#pragma unroll
    for (int k = 0; k < kAhead; k++) {
        const int c = group + k * kShares;
        ahead[k] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        if (c < a.chunks) ahead[k] = at.o_at(c, d);
    }
    const int sid = a.bt.seq ? gld(a.bt.seq + b) : b;
    if (sid < 0 || sid >= a.kv.seqs) return;
    const Span sp = span_of(a, static_cast<int>(kv_len_of(a.kv, sid)), kv_rows_of(a.bt.n_new, b, a.bt.M));
    if (r >= sp.n * a.group) return;
    const int n = chunks_of(a, sp);
    float top = tid < n ? m_ahead : -INFINITY;
    for (int c = tid + threads; c < n; c += threads) top = fmaxf(top, at.m_at(c));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if ((tid & 63) == 0) s_top[tid >> 6] = top;
    __syncthreads();
    for (int i = 0; i < threads / 64; i++) top = fmaxf(top, s_top[i]);
    f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
    // its share: that of the places loaded ahead, which past the sinks are
    // `jump - first` ahead of their index
    const int share = (group + (sp.jump - sp.first)) % kShares;
    if (top == -INFINITY) top = 0.0f;  // nothing visible, or only NaN: the sums are 0, or NaN
    for (int from = 0; from < n; from += kWeights) {
        const int upto = min(n - from, kWeights);
        for (int i = tid; i < upto; i += threads) {
            const bool held = from + i == tid;
            const float w = __builtin_amdgcn_exp2f((held ? m_ahead : at.m_at(from + i)) - top);
            s_w[i] = w;
            s_wl[i] = w * (held ? l_ahead : at.l_at(from + i));
        }
        __syncthreads();
        for (int nth = 0; nth < 2; nth++) {
            const Run run(sp, n, nth);
            const int lo = max(run.from, from), hi = min(run.to, from + upto);
            int c = lo + ((share - (lo + run.shift)) % kShares + kShares) % kShares;
#pragma unroll
            for (int k = 0; k < kAhead; k++)
                if (c == group + k * kShares && c < hi) {
                    v += s_w[c - from] * ahead[k];
                    l += s_wl[c - from];
                    c += kShares;
                }
#pragma unroll 4
            for (; c < hi; c += kShares) {
                v += s_w[c - from] * at.o_at(c, d);
                l += s_wl[c - from];
            }
        }
        __syncthreads();
    }
    *reinterpret_cast<f4 *>(s_v + share * D + d) = v;
    if (d == 0) s_l[share] = l;
    __syncthreads();
    f4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    float sum = 0.0f;
    if (tid < quads) {
        for (int i = 0; i < kShares; i++) {
            x += *reinterpret_cast<f4 *>(s_v + i * D + 4 * tid);
            sum += s_l[i];
        }
        if (tid == 0) flag_over(a, sp);
        // its own place in the first share's sums
        *reinterpret_cast<f4 *>(s_v + 4 * tid) = joined(a, sp, x, sum);
    }
    __syncthreads();
    finish_rows(a, s_v, D, b, head, r, 1);
}

// Many rows: dim / 4 threads each, which hold the shares' sums in registers.
__global__ __launch_bounds__(kJoin) void kv_attn_join_rows_kernel(AttnArgs a) {
    __shared__ __align__(16) float s_v[kJoin * 4];
    fetch_args<sizeof(AttnArgs)>();
    const int D = a.kv.dim, quads = D / 4, of = kJoin / quads;
    const int head = blockIdx.y, b = blockIdx.z, row0 = blockIdx.x * of, tid = threadIdx.x;
    const int i = tid / quads, d = (tid - i * quads) * 4, r = row0 + min(i, of - 1);
    const Parts at(a, b, head, min(r, a.rows - 1));
    float m[kAhead];
#pragma unroll
    for (int c = 0; c < kAhead; c++) m[c] = c < a.chunks ? at.m_at(c) : 0.0f;
    const int sid = a.bt.seq ? gld(a.bt.seq + b) : b;
    if (sid < 0 || sid >= a.kv.seqs) return;
    const Span sp = span_of(a, static_cast<int>(kv_len_of(a.kv, sid)), kv_rows_of(a.bt.n_new, b, a.bt.M));
    const int rows = min(sp.n * a.group - row0, of);
    if (rows <= 0) return;
    const int n = chunks_of(a, sp);
    if (i < rows) {
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kAhead; c++) top = c < n ? fmaxf(top, m[c]) : top;
#pragma unroll 8
        for (int c = kAhead; c < n; c++) top = fmaxf(top, at.m_at(c));
        f4 v[kShares];
        float s[kShares];
#pragma unroll
        for (int k = 0; k < kShares; k++) {
            v[k] = f4{0.0f, 0.0f, 0.0f, 0.0f};
            s[k] = 0.0f;
        }
        if (top == -INFINITY) top = 0.0f;  // as above
        for (int nth = 0; nth < 2; nth++) {
            const Run run(sp, n, nth);
            // rounds of one chunk of each share
            for (int c0 = run.from - ((run.from + run.shift) & (kShares - 1)); c0 < run.to; c0 += kShares) {
                f4 o[kShares];
                float mc[kShares], lc[kShares];
#pragma unroll
                for (int k = 0; k < kShares; k++) {
                    const int c = c0 + k;
                    const bool in = c >= run.from && c < run.to;
                    o[k] = in ? at.o_at(c, d) : f4{0.0f, 0.0f, 0.0f, 0.0f};
                    mc[k] = in ? at.m_at(c) : -INFINITY;
                    lc[k] = in ? at.l_at(c) : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < kShares; k++) {
                    const float w = __builtin_amdgcn_exp2f(mc[k] - top);
                    v[k] += w * o[k];
                    s[k] += w * lc[k];
                }
            }
        }
        f4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kShares; k++) {
            x += v[k];
            sum += s[k];
        }
        if (i == 0 && d == 0) flag_over(a, sp);
        *reinterpret_cast<f4 *>(s_v + i * D + d) = joined(a, sp, x, sum);
    }
    __syncthreads();
    finish_rows(a, s_v, D, b, head, row0, rows);
}

// Rows from which the second kernel is taken: with ten workgroups of one row
// to a compute unit (us: 3200 rows of 128 in 13 chunks 10.5 against 8.0, 2048
// rows of 64 in 22 chunks 8.4 against 9.0; these two differ in dim and chunks
// as well, and nothing between them was measured).
constexpr int64_t kManyRows = 2560;

// Chunks that a sequence can have: of its whole length, or of what a window
// and the sinks can touch.
static int64_t chunks_within(int64_t bound, int64_t window, int64_t sinks, int64_t chunk) {
    const int64_t all = (bound + chunk - 1) / chunk;
    if (!window) return all;
    const int64_t most = (sinks + chunk - 1) / chunk + (window + SV_MAX_M + chunk - 1) / chunk + 1;
    return std::min(all, most);
}

// Slots of a chunk when the caller leaves the choice: the shortest with which
// the launch is one round of workgroups (256 compute units hold two each), for
// sequences of the length that max_len, or else the table row, allows.  Far
// shorter ones leave most of the chip idle: 4099 slots take 17.3 us with their
// own length as max_len, and 40.6 in a table row of 131072 without it.
// Without a window the sequences of a batch are seldom all as long as the
// longest: half a round more is allowed for.  Past one round of 2048, chunks
// short enough to even out the last round (two cases, the last ones below).
// Measured in us, heads of 128 and groups of 5 where nothing else is said:
//   5 x 4099 slots, 8 heads, fp16          128: 20, 256: 17, 384: 21
//   8 rows, window 1024, 8 heads of 96     128: 16, 256: 16, 512: 18
//   4 trees of up to 8191, 8 heads of 64   256: 33, 384: 25, 512: 28
//   16 sequences up to 16384, int8         1024: 85, 1280: 80, 2048: 92
//   32 sequences, window 4096, fp16        1024: 125, 1280: 123, 2048: 132
// A sequence that fits one short chunk needs no join (300 slots: 9.7 us
// against 11.8 with chunks of 256).
static int chunk_rule(int64_t pairs, bool batch, int64_t bound, int64_t window, int64_t sinks) {
    if (bound <= 512) return static_cast<int>((bound + 127) / 128 * 128);
    const int64_t room = batch && !window ? 768 : 512;
    for (int c = 256; c <= 2048; c += 128) {
        // of a window that lies anywhere: window / c + 1 chunks on average
        const int64_t units = window && window + sinks < bound ? pairs * ((sinks + c - 1) / c + 1) + pairs * window / c
                                                               : pairs * ((bound + c - 1) / c);
        if (units <= room) return c;
    }
    int c = 1280;  // and of a pool of very long sequences, no more than 2^17
    while (c < (1 << 23) && pairs * chunks_within(bound, window, sinks, c) > (1 << 17)) c *= 2;
    return c;
}

// The time of a launch, for the choice of its chunks where slots are shared.  A
// unit of work takes kUnit for its start and end, and a time for each slot of
// its row group.  Shared chunks come first; the sequences' own ones fill the
// last round.  Half a round or less is faster, where it leaves each wave a SIMD
// of its own.  Fitted to sweeps of the chunk length (us, fp16, 16 sequences of
// 5 x 5 rows of 128 and 8 heads, 32768 shared slots in chunks of 8192, 4096,
// 2048, 1280: 136, 145, 147, 162; bf16, 32 sequences of 5 rows, 16384 slots in
// chunks of 4096, 2048, 1024: 94, 58, 66).
constexpr double kUnit = 10.0, kJoinBytes = 4e6;  // us; bytes of partial sums a us
struct Load {
    double slot;    // us
    int64_t round;  // workgroups that the chip holds: of four waves two a compute unit, of two four or (LDS) two
    Load(int type, int dim, int rt) {
        const bool four = type == SV_KV_I8 || (type == SV_KV_F16 && dim <= 128);
        round = four || dim > 128 ? 512 : 1024;
        slot = 0.0149 * (0.3 + 0.7 * dim / 128) * (0.35 + 0.325 * rt) * (type == SV_KV_I8 ? 1.4 : four ? 1.0 : 2.1);
    }
    // n1 units of c1 slots, then n2 of c2
    double time(int64_t n1, int64_t c1, int64_t n2, int64_t c2) const {
        const double l1 = kUnit + slot * c1, l2 = kUnit + slot * c2;
        auto part = [&](int64_t m) { return m == 0 ? 0.0 : m <= round / 2 ? 0.62 : 1.0; };
        const int64_t left = n1 % round;
        double t = l1 * (n1 / round + (left ? part(left + n2) : 0.0)), over = n2 * l2 - (left ? (round - left) * l1 : 0.0);
        if (over > 0.0) t += std::max(over / round, n1 ? 0.0 : l2 * part(n2 % round));
        return t;
    }
};

// Slots of a chunk where the first `shared` of up to `bound` are to be read
// once for the rows of all B sequences, in `tiles` row groups and not in
// own_tiles for each sequence; 0 where that gains nothing over `plain` slots a
// chunk without it.  A shared unit takes some 3 us more (positions and tables
// of several sequences).  us, shared against not: 32 sequences of 5 rows, 16384
// slots, bf16 58 against 228; 8 trees of 16 x 4 rows of 64, 8000 slots, int8,
// whose tiles are full either way 46 against 45; 4 x 5 rows, 960 slots 15
// against 13.  The sequences' own chunks are counted in own_tiles row groups too,
// though bf16 is launched with groups half as tall (from 17 rows on, 33 up to 64
// of dim): counted as launched, the choice differs in 31 of 4000 drawn shapes,
// which then take 1195 us together and not 1122 (15 x 24 rows of 96, 2048 slots
// 38 against 30; but 4 x 64 rows of 96, 18368 slots 37 against 43).
static int chunk_rule_shared(const KvDev &d, int64_t B, int64_t rows, int rt, int64_t tiles, int own_rt, int64_t own_tiles,
                             int64_t bound, int64_t shared, int plain) {
    const double row_bytes = static_cast<double>(d.blk_bytes) / kBlk, parts = static_cast<double>(B) * d.heads * rows * d.dim * 8;
    const int64_t chunks = (bound + plain - 1) / plain, units = B * d.heads * own_tiles * chunks;
    double best = Load(d.type, d.dim, own_rt).time(0, 0, units, std::min<int64_t>(plain, bound)) + chunks * parts / kJoinBytes;
    best = std::max(best, B * d.heads * static_cast<double>(bound) * row_bytes / 6.5e6);
    const Load load(d.type, d.dim, rt);
    int64_t chosen = 0;
    for (int64_t n = 1; n <= 48; n++) {
        const int64_t c = shared / n / 128 * 128, rest = bound - n * c;
        if (c < 256) break;
        if (c > (1 << 23)) continue;
        const int64_t own = (rest + c - 1) / c;
        const double t = load.time(d.heads * tiles * n, c, B * d.heads * own_tiles * own, std::min(rest, c)) + 3.0 +
                         (n + own) * parts / kJoinBytes;
        if (t < best) {
            best = t;
            chosen = c;
        }
    }
    return static_cast<int>(chosen);
}

struct Plan {
    int64_t bound, units;
    int rt;
    size_t o_m, o_l, bytes;
};

static int plan_of(const KvDev &d, const sv_kv_batch *bt, const sv_kv_attn *at, int64_t shared, AttnShared *a, Plan *p) {
    SV_REQUIRE(at, SV_ERR_ARG, "kv_attention: NULL arguments");
    SV_REQUIRE(at->q_heads >= 1 && at->q_heads % d.heads == 0 && at->q_heads / d.heads <= 64, SV_ERR_SHAPE,
               "kv_attention: q_heads must be a multiple of heads, at most 64 times");
    SV_REQUIRE(at->scale > 0.0f && at->scale <= 2.3e38f, SV_ERR_ARG,
               "kv_attention: scale must be positive and at most 2.3e38");  // times log2(e) it is finite
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
    a->scale = at->scale * 1.44269504088896340736f;
    SV_REQUIRE(shared >= 0 && shared <= cap, SV_ERR_ARG, "kv_attention: shared must be in [0, width * page]");
    SV_REQUIRE(shared == 0 || at->window == 0, SV_ERR_ARG, "kv_attention: a window and shared slots do not go together");
    shared = std::min(shared, p->bound);
    const int64_t all_rows = static_cast<int64_t>(bt->B) * a->rows;
    const int own_rt = attn_tiles_per_wave(d.dim, a->rows);
    int rt = attn_tiles_shared(d.type, d.dim, static_cast<int>(all_rows));
    auto tiles_of = [](int64_t rows, int rt) { return (rows + 16 * rt - 1) / (16 * rt); };
    a->chunk = at->chunk;
    if (!a->chunk) {
        a->chunk = chunk_rule(static_cast<int64_t>(bt->B) * d.heads, bt->B > 1, p->bound, at->window, at->sinks);
        if (shared >= 256 && bt->B > 1) {
            const int c = chunk_rule_shared(d, bt->B, a->rows, rt, tiles_of(all_rows, rt), own_rt, tiles_of(a->rows, own_rt),
                                            p->bound, shared, a->chunk);
            if (c) a->chunk = c;
            else shared = 0;
        }
    }
    const int64_t chunks = chunks_within(p->bound, at->window, at->sinks, a->chunk);
    a->chunks = static_cast<int32_t>(chunks);
    // one sequence, or one chunk, shares nothing
    a->shared = bt->B > 1 && chunks > 1 ? static_cast<int32_t>(shared / a->chunk) : 0;
    if (!a->shared) rt = own_rt;
    p->rt = rt;
    a->tiles = static_cast<int32_t>(tiles_of(a->rows, rt));
    a->shared_tiles = static_cast<int32_t>(tiles_of(all_rows, rt));
    const int64_t shared_grid = (static_cast<int64_t>(a->shared) * d.heads + 7) / 8 * 8 * a->shared_tiles;
    SV_REQUIRE(shared_grid < (1ll << 23), SV_ERR_SHAPE, "kv_attention: too many chunks (use a longer chunk)");
    a->shared_grid = static_cast<int32_t>(shared_grid);
    a->by_rows = div_by(a->rows);
    a->by_m = div_by(bt->M);
    a->by_shared_tiles = div_by(a->shared_tiles);
    a->by_group = div_by(a->group);
    a->by_chunk = div_by(a->chunk);
    a->by_tiles = div_by(a->tiles);
    a->by_heads = div_by(d.heads);
    a->by_turns = div_by(std::max(1, a->rope.rot / 8));
    p->units = static_cast<int64_t>(bt->B) * d.heads * (chunks - a->shared);
    SV_REQUIRE(p->units * a->tiles < (1ll << 23), SV_ERR_SHAPE, "kv_attention: too many chunks (use a longer chunk)");
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

extern "C" size_t sv_kv_attention_shared_workspace_bytes(const sv_kv *kv, const sv_kv_batch *batch, const sv_kv_attn *attn,
                                                         int32_t shared) {
    KvDev d;
    AttnShared a{};
    Plan p;
    if (kv_check(kv, "kv_attention", &d) || kv_check_batch(d, batch, "kv_attention", SV_MAX_M) ||
        plan_of(d, batch, attn, shared, &a, &p))
        return 0;
    return p.bytes;
}

extern "C" size_t sv_kv_attention_workspace_bytes(const sv_kv *kv, const sv_kv_batch *batch, const sv_kv_attn *attn) {
    return sv_kv_attention_shared_workspace_bytes(kv, batch, attn, 0);
}

extern "C" int sv_kv_attention(const sv_kv *kv, int32_t layer, const sv_kv_batch *batch, const sv_kv_attn *attn,
                               const float *q, float *out, const sv_epilogue *ep, void *workspace, size_t ws_bytes,
                               void *stream) {
    return sv_kv_attention_shared(kv, layer, batch, attn, 0, q, out, ep, workspace, ws_bytes, stream);
}

extern "C" int sv_kv_attention_shared(const sv_kv *kv, int32_t layer, const sv_kv_batch *batch, const sv_kv_attn *attn,
                                      int32_t shared, const float *q, float *out, const sv_epilogue *ep, void *workspace,
                                      size_t ws_bytes, void *stream) {
    KvDev d;
    AttnShared a{};
    Plan p;
    int rc = kv_check(kv, "kv_attention", &d);
    if (!rc) rc = kv_check_batch(d, batch, "kv_attention", SV_MAX_M);
    if (!rc) rc = plan_of(d, batch, attn, shared, &a, &p);
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
    auto launch = [&](const auto &args) {
        return d.type == SV_KV_F16    ? attn_launch_f16(args, p.rt, p.units, st)
               : d.type == SV_KV_BF16 ? attn_launch_bf16(args, p.rt, p.units, st)
                                      : attn_launch_i8(args, p.rt, p.units, st);
    };
    rc = a.shared ? launch(a) : launch(static_cast<const AttnArgs &>(a));
    if (rc || a.chunks == 1) return rc;
    const int of = kJoin / (d.dim / 4);
    if (static_cast<int64_t>(a.rows) * d.heads * batch->B >= kManyRows)
        hipLaunchKernelGGL(kv_attn_join_rows_kernel, dim3((a.rows + of - 1) / of, d.heads, batch->B), dim3(kJoin), 0, st, static_cast<const AttnArgs &>(a));
    else
        hipLaunchKernelGGL(kv_attn_join_kernel, dim3(a.rows, d.heads, batch->B), dim3(kShares * (d.dim / 4)), 0, st,
                           static_cast<const AttnArgs &>(a));
    return hip_check(hipGetLastError(), "kv_attention join launch");
}
