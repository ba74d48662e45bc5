// kv.hip - key-value cache: rows written and read, and the page operators.
//
// The page operators' bookkeeping (free list, holders, tables, lengths) is a
// few hundred words per call, so each runs in one workgroup of 16 waves: a
// wave takes a sequence's table row 64 entries at a time, and the order in
// which pages leave or join the free list is fixed by a prefix sum over the
// sequences, never by the order in which waves run.  What moves data is a
// launch of its own behind it, over all layers and heads.
#include "kv_internal.h"

namespace sv {

static int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) s++;
    return s;
}

static bool kv_shape_ok(int32_t type, int32_t heads, int32_t dim, int32_t page) {
    if (type != SV_KV_F16 && type != SV_KV_BF16 && type != SV_KV_I8) return false;
    if (heads < 1 || heads > kKvMaxHeads || dim < 32 || dim > kMaxDim || dim % 32) return false;
    return page == 32 || page == 64 || page == 128 || page == 256;
}

int kv_check(const sv_kv *kv, const char *who_, KvDev *o) {
    const std::string who(who_);
    SV_REQUIRE(kv, SV_ERR_ARG, who + ": NULL cache");
    SV_REQUIRE(kv->type == SV_KV_F16 || kv->type == SV_KV_BF16 || kv->type == SV_KV_I8, SV_ERR_QTYPE,
               who + ": unsupported cache type");
    SV_REQUIRE(kv_shape_ok(kv->type, kv->heads, kv->dim, kv->page), SV_ERR_SHAPE,
               who + ": heads must be in [1, 4096], dim a multiple of 32 up to 256, page 32, 64, 128 or 256");
    SV_REQUIRE(kv->layers >= 1 && kv->layers <= kKvMaxLayers &&
                   static_cast<int64_t>(kv->layers) * kv->heads < (1 << 23),
               SV_ERR_SHAPE, who + ": layers must be in [1, 4096], layers * heads below 2^23");
    SV_REQUIRE(kv->n_pages >= 1 && kv->n_pages <= kKvMaxPages, SV_ERR_SHAPE, who + ": n_pages must be in [1, 2^24]");
    SV_REQUIRE(sv_kv_data_bytes(kv), SV_ERR_SHAPE, who + ": the pool must be below 2^48 bytes");
    SV_REQUIRE(kv->seqs >= 1 && kv->seqs <= SV_KV_MAX_SEQS && kv->width >= 1 &&
                   static_cast<int64_t>(kv->seqs) * kv->width < (1ll << 31) &&
                   static_cast<int64_t>(kv->width) * kv->page < (1ll << 31) - 65536,
               SV_ERR_SHAPE, who + ": seqs must be in [1, 4096], seqs * width and width * page below 2^31");
    SV_REQUIRE(kv->data && kv->table && kv->len && kv->refs && kv->free_ids && kv->ctl, SV_ERR_ARG,
               who + ": NULL cache buffer");
    SV_REQUIRE(aligned(kv->data, 256), SV_ERR_ALIGN, who + ": the pool must be 256-byte aligned");
    SV_REQUIRE(aligned(kv->table, 4) && aligned(kv->len, 4) && aligned(kv->refs, 4) && aligned(kv->free_ids, 4) &&
                   aligned(kv->ctl, 4),
               SV_ERR_ALIGN, who + ": int32 buffers must be 4-byte aligned");
    o->data = static_cast<uint8_t *>(kv->data);
    o->table = kv->table;
    o->len = kv->len;
    o->refs = kv->refs;
    o->free_ids = kv->free_ids;
    o->ctl = kv->ctl;
    o->type = kv->type;
    o->layers = kv->layers;
    o->heads = kv->heads;
    o->dim = kv->dim;
    o->n_pages = kv->n_pages;
    o->seqs = kv->seqs;
    o->width = kv->width;
    o->page = kv->page;
    o->page_shift = log2_of(kv->page);
    o->blk_shift = o->page_shift - 5;
    o->blk_bytes = kv_block_bytes(kv->type, kv->dim);
    o->page_bytes = static_cast<int64_t>(sv_kv_page_bytes(kv->type, kv->heads, kv->dim, kv->page));
    return SV_OK;
}

int kv_check_batch(const KvDev &kv, const sv_kv_batch *b, const char *who_, int max_m) {
    const std::string who(who_);
    SV_REQUIRE(b, SV_ERR_ARG, who + ": NULL batch");
    SV_REQUIRE(b->B >= 1 && b->B <= SV_KV_MAX_SEQS, SV_ERR_ARG, who + ": B must be in [1, 4096]");
    SV_REQUIRE(b->seq || b->B <= kv.seqs, SV_ERR_ARG, who + ": B exceeds the cache's sequences");
    SV_REQUIRE(b->M >= 1 && b->M <= max_m, SV_ERR_ARG, who + ": M must be in [1, " + std::to_string(max_m) + "]");
    SV_REQUIRE(!b->tree || b->M <= 32, SV_ERR_ARG, who + ": tree masks need M <= 32");
    SV_REQUIRE((!b->seq || aligned(b->seq, 4)) && (!b->n_new || aligned(b->n_new, 4)) &&
                   (!b->tree || aligned(b->tree, 4)),
               SV_ERR_ALIGN, who + ": int32 buffers must be 4-byte aligned");
    return SV_OK;
}

int kv_check_rope(const KvDev &kv, const sv_kv_rope *r, const char *who_) {
    const std::string who(who_);
    if (!r || r->mode == SV_ROPE_NONE) return SV_OK;
    SV_REQUIRE(r->mode == SV_ROPE_PAIRS || r->mode == SV_ROPE_HALVES, SV_ERR_ARG, who + ": unknown rope mode");
    SV_REQUIRE(r->rot >= 2 && r->rot % 2 == 0 && r->rot <= kv.dim, SV_ERR_SHAPE,
               who + ": rope.rot must be even and at most dim");
    SV_REQUIRE(static_cast<int64_t>(r->n_pos) >= static_cast<int64_t>(kv.width) * kv.page, SV_ERR_SHAPE,
               who + ": the rope table must cover width * page positions");
    SV_REQUIRE(r->table, SV_ERR_ARG, who + ": NULL rope table");
    SV_REQUIRE(aligned(r->table, 16), SV_ERR_ALIGN, who + ": the rope table must be 16-byte aligned");
    return SV_OK;
}

// ------------------------------------------------------------ bookkeeping
constexpr int kBookThreads = 1024, kBookWaves = 16;

// Exclusive prefix sum of cnt[0..n) in place (LDS); returns the total.  All
// threads of the workgroup take part.
__device__ int scan_counts(int *cnt, int n) {
    __shared__ int wsum[kBookWaves + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int run = 0;
    for (int at = 0; at < n; at += kBookThreads) {
        const int i = at + tid;
        const int own = i < n ? cnt[i] : 0;
        int v = own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int t = __shfl_up(v, o, 64);
            if (lane >= o) v += t;
        }
        __syncthreads();
        if (lane == 63) wsum[wave] = v;
        __syncthreads();
        int before = run, all = 0;
        for (int w = 0; w < kBookWaves; w++) {
            if (w < wave) before += wsum[w];
            all += wsum[w];
        }
        if (i < n) cnt[i] = before + v - own;
        run += all;
    }
    __syncthreads();
    return run;
}

// The table row of place b of a list, or -1 where it is out of range or an
// earlier place names it.  Called by a whole wave.
__device__ int first_sid(const int32_t *seq, int b, int seqs) {
    if (!seq) return b < seqs ? b : -1;
    const int sid = gld(seq + b), lane = threadIdx.x & 63;
    if (sid < 0 || sid >= seqs) return -1;
    for (int at = 0; at < b; at += 64) {
        const int j = at + lane;
        if (__any(j < b && gld(seq + j) == sid)) return -1;
    }
    return sid;
}

__device__ __forceinline__ int lane_rank(unsigned long long mask) {
    return __popcll(mask & ((1ull << (threadIdx.x & 63)) - 1));
}

__global__ __launch_bounds__(kBookThreads) void kv_init_kernel(KvDev kv) {
    fetch_args<sizeof(KvDev)>();
    const int64_t n = static_cast<int64_t>(kv.seqs) * kv.width;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kBookThreads;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kBookThreads + threadIdx.x;
    for (int64_t i = at; i < n; i += step) gst(kv.table + i, -1);
    for (int64_t i = at; i < kv.seqs; i += step) gst(kv.len + i, 0);
    for (int64_t i = at; i < kv.n_pages; i += step) {
        gst(kv.refs + i, 0);
        gst(kv.free_ids + i, static_cast<int32_t>(kv.n_pages - 1 - i));
    }
    if (at < 4) gst(kv.ctl + at, at == 0 ? kv.n_pages : 0);
}

// A wave's share of a reservation: the entries of place b that lack a page.
// pass 0 returns how many there are; pass 1 fills them, the first of them
// from free_ids[top], the next ones below it.
__device__ int reserve_row(const KvDev &kv, const sv_kv_batch &bt, int b, bool fill, int top, int *over) {
    const int lane = threadIdx.x & 63, sid = first_sid(bt.seq, b, kv.seqs);
    if (sid < 0) return 0;
    const int64_t len = kv_len_of(kv, sid);
    const int64_t lo = (len + kv.page - 1) >> kv.page_shift;
    int64_t hi = (len + kv_rows_of(bt.n_new, b, bt.M) + kv.page - 1) >> kv.page_shift;
    if (hi > kv.width) {
        *over = 1;
        hi = kv.width;
    }
    int have = 0;
    for (int64_t at = lo; at < hi; at += 64) {
        int32_t *p = kv.table + static_cast<int64_t>(sid) * kv.width + at + lane;
        const bool want = at + lane < hi && gld(p) < 0;
        const unsigned long long m = __ballot(want);
        if (fill && want) {
            const int page = gld(kv.free_ids + (top - have - lane_rank(m)));
            if (page >= 0 && page < kv.n_pages) {
                gst(p, page);
                gst(kv.refs + page, 1);
            }
        }
        have += __popcll(m);
    }
    return have;
}

__global__ __launch_bounds__(kBookThreads) void kv_reserve_kernel(KvDev kv, sv_kv_batch bt) {
    fetch_args<sizeof(KvDev) + sizeof(sv_kv_batch)>();
    __shared__ int cnt[SV_KV_MAX_SEQS];
    __shared__ int over;
    const int tid = threadIdx.x, wave = tid >> 6;
    if (tid == 0) over = 0;
    __syncthreads();
    const int fc = min(max(gld(kv.ctl), 0), kv.n_pages);
    for (int b = wave; b < bt.B; b += kBookWaves) {
        const int have = reserve_row(kv, bt, b, false, 0, &over);
        if ((tid & 63) == 0) cnt[b] = have;
    }
    __syncthreads();
    const int total = scan_counts(cnt, bt.B);
    if (over || total > fc) {
        if (tid == 0) kv_flag(kv, over ? SV_KV_TOO_LONG : SV_KV_NO_PAGES);
        return;
    }
    if (total == 0) return;
    for (int b = wave; b < bt.B; b += kBookWaves) reserve_row(kv, bt, b, true, fc - 1 - cnt[b], &over);
    __syncthreads();
    if (tid == 0) gst(kv.ctl, fc - total);
}

// Takes the entries [from[b], width) off the table rows of a list.  A page
// that no row holds any more goes on the free list, in the order of the last
// entry naming it (places of the list in order, then entries): all entries
// give up their hold, then each entry of a page without holders claims it by
// an atomic minimum of -(1 + order), so which claim wins does not depend on
// timing.  The callers clear cnt[SV_KV_MAX_SEQS] ahead of a barrier: whether
// there is an entry at all, later the pages freed.
constexpr int kSkip = 0x7FFFFFFF;
__device__ void drop_pages(const KvDev &kv, const int32_t *seq, int n, const int *from, int *cnt) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int fc = min(max(ld_dev(kv.ctl), 0), kv.n_pages);  // until the last store below
    int held = -1;  // the first entry of the lane, read once: only its own wave changes it
    for (int pass = 0; pass < 4; pass++) {
        for (int b = wave; b < n; b += kBookWaves) {
            int have = pass == 3 ? cnt[b] : 0;
            if (from[b] != kSkip) {
                const int sid = seq ? gld(seq + b) : b;
                int32_t *row = kv.table + static_cast<int64_t>(sid) * kv.width;
                for (int64_t at = from[b]; at < kv.width; at += 64) {
                    const int64_t e = at + lane;
                    const bool first = b == wave && at == from[b];
                    int page = held;
                    if (!first || pass == 0) page = e < kv.width ? gld(row + e) : -1;
                    if (first) held = page;
                    if (!__any(page >= 0)) break;  // a row's pages come first
                    if (pass == 0 && lane == 0) cnt[SV_KV_MAX_SEQS] = 1;
                    const bool ok = page >= 0 && page < kv.n_pages;
                    const int claim = -1 - static_cast<int>(static_cast<int64_t>(b) * kv.width + e);
                    if (pass == 0) {
                        if (ok) add_dev(kv.refs + page, -1);
                    } else if (pass == 1) {
                        if (ok && ld_dev(kv.refs + page) <= 0)
                            __hip_atomic_fetch_min((SV_GLOBAL int32_t *)(kv.refs + page), claim, __ATOMIC_RELAXED,
                                                   __HIP_MEMORY_SCOPE_AGENT);
                    } else {
                        const bool push = ok && ld_dev(kv.refs + page) == claim;
                        const unsigned long long m = __ballot(push);
                        if (pass == 3) {
                            const int to = fc + have + lane_rank(m);
                            if (push && to < kv.n_pages) {
                                gst(kv.free_ids + to, page);
                                st_dev(kv.refs + page, 0);
                            }
                            if (page >= 0) gst(row + e, -1);
                        }
                        have += __popcll(m);
                    }
                }
            }
            if (pass == 2 && lane == 0) cnt[b] = have;
        }
        drain();
        __syncthreads();
        if (pass == 0 && cnt[SV_KV_MAX_SEQS] == 0) return;  // most commits leave no page to drop: 4.6 -> 2.9 us
        if (pass == 2) {
            const int total = scan_counts(cnt, n);
            // pass 3 reads the old count before anyone stores the new one
            if (tid == 0) cnt[SV_KV_MAX_SEQS] = total;
            __syncthreads();
        }
    }
    if (tid == 0) st_dev(kv.ctl, min(fc + cnt[SV_KV_MAX_SEQS], kv.n_pages));
}

__global__ __launch_bounds__(kBookThreads) void kv_release_kernel(KvDev kv, const int32_t *ids, int n) {
    fetch_args<sizeof(KvDev) + 16>();
    __shared__ int from[SV_KV_MAX_SEQS];
    __shared__ int cnt[SV_KV_MAX_SEQS + 1];
    if (threadIdx.x == 0) cnt[SV_KV_MAX_SEQS] = 0;
    for (int b = threadIdx.x >> 6; b < n; b += kBookWaves) {
        const int sid = first_sid(ids, b, kv.seqs);
        if ((threadIdx.x & 63) == 0) {
            from[b] = sid < 0 ? kSkip : 0;
            if (sid >= 0) gst(kv.len + sid, 0);
        }
    }
    __syncthreads();
    drop_pages(kv, ids, n, from, cnt);
}

// Whether place b's count and path can be kept; the rows kept, 0 for a
// failed round, -1 if it is refused.  Called by a whole wave; r is the row
// that the path gives the lane's place (M <= 32 with a path).
__device__ int kept_rows(const sv_kv_batch &bt, const int32_t *accepted, int stride, const int32_t *path, int b,
                         int *row = nullptr) {
    const int lane = threadIdx.x & 63;
    const int r = path && lane < bt.M ? gld(path + static_cast<int64_t>(b) * bt.M + lane) : lane;
    const int a = gld(accepted + static_cast<int64_t>(b) * stride), n = kv_rows_of(bt.n_new, b, bt.M);
    const int before = __shfl_up(r, 1);
    if (row) *row = r;
    if (a < 0) return 0;
    if (a >= n) return -1;
    if (path && __any(lane <= a && (r >= n || r <= (lane ? before : -1)))) return -1;
    return a + 1;
}

__global__ __launch_bounds__(kBookThreads) void kv_commit_kernel(KvDev kv, sv_kv_batch bt, const int32_t *accepted,
                                                                 int stride, const int32_t *path) {
    fetch_args<sizeof(KvDev) + sizeof(sv_kv_batch) + 24>();
    __shared__ int from[SV_KV_MAX_SEQS];
    __shared__ int cnt[SV_KV_MAX_SEQS + 1];
    if (threadIdx.x == 0) cnt[SV_KV_MAX_SEQS] = 0;
    const int64_t cap = static_cast<int64_t>(kv.width) * kv.page;
    for (int b = threadIdx.x >> 6; b < bt.B; b += kBookWaves) {
        int row = 0;
        const int sid = first_sid(bt.seq, b, kv.seqs), kept = kept_rows(bt, accepted, stride, path, b, &row);
        const int last = path ? __shfl(row, max(kept, 1) - 1) : kept - 1;  // the last row kept
        if ((threadIdx.x & 63) == 0) {
            from[b] = kSkip;
            if (sid >= 0) {
                // a row that append dropped, for want of a page, is not kept
                const int64_t old = kv_len_of(kv, sid), len = old + kept;
                if (kept < 0 || len > cap ||
                    (kept > 0 && (kv_page_of(kv, sid, (len - 1) >> kv.page_shift) < 0 ||
                                  kv_page_of(kv, sid, (old + last) >> kv.page_shift) < 0))) {
                    kv_flag(kv, SV_KV_BAD_COMMIT);
                } else {
                    gst(kv.len + sid, static_cast<int32_t>(len));
                    from[b] = static_cast<int>((len + kv.page - 1) >> kv.page_shift);
                }
            }
        }
    }
    __syncthreads();
    drop_pages(kv, bt.seq, bt.B, from, cnt);
}

// Moves the kept rows of a tree together, before the bookkeeping: a
// workgroup per (head and layer, sequence).  Row path[i] >= i moves to slot
// len + i, and one thread moves one element of every row, eight rows at a
// time in ascending order: all are read before any is written, and what
// later rows are read from lies behind what was written.  Bound by latency
// (the path, the pages and the rows are loads that wait for one another); the
// moved rows are a few KB.  Row by row it took 20.8 us where this takes
// 12.2 (4 sequences of 64 layers and 8 heads, 6 rows each).
struct Move {
    const uint8_t *from;  // blocks
    uint8_t *to;
    int k0, k1;           // slots in them
};
template <typename T, typename F>
__device__ __forceinline__ void move_all(const Move *moves, int n, F at) {
    for (int i0 = 0; i0 < n; i0 += 8) {
        T x[8];
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (i0 + k < n) x[k] = gld(reinterpret_cast<const T *>(moves[i0 + k].from + at(moves[i0 + k].k0)));
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (i0 + k < n) gst(reinterpret_cast<T *>(moves[i0 + k].to + at(moves[i0 + k].k1)), x[k]);
    }
}
__global__ __launch_bounds__(256) void kv_commit_move_kernel(KvDev kv, sv_kv_batch bt, const int32_t *accepted,
                                                             int stride, const int32_t *path) {
    fetch_args<sizeof(KvDev) + sizeof(sv_kv_batch) + 24>();
    __shared__ int s_n;
    __shared__ Move moves[32];
    const int b = blockIdx.y, head = blockIdx.x % kv.heads, layer = blockIdx.x / kv.heads;
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int row = 0, n = 0;
        const int kept = kept_rows(bt, accepted, stride, path, b, &row), sid = first_sid(bt.seq, b, kv.seqs);
        if (kept > 0 && sid >= 0) {
            const int64_t len = kv_len_of(kv, sid), s0 = len + row, s1 = len + lane;
            const bool own = lane < kept;
            const int p0 = own ? kv_page_of(kv, sid, s0 >> kv.page_shift) : -1;
            const int p1 = own ? kv_page_of(kv, sid, s1 >> kv.page_shift) : -1;
            // the bookkeeping refuses what does not fit; nothing moves then
            const bool ok = len + kept <= static_cast<int64_t>(kv.width) * kv.page && __shfl(p0, kept - 1) >= 0 &&
                            __shfl(p1, kept - 1) >= 0;
            const bool moved = ok && own && row != lane && p0 >= 0 && p1 >= 0;
            const unsigned long long m = __ballot(moved);
            n = __popcll(m);
            if (moved)
                moves[lane_rank(m)] = Move{kv_block(kv, layer, p0, head, static_cast<int>(s0 & (kv.page - 1)) >> 5),
                                           kv_block(kv, layer, p1, head, static_cast<int>(s1 & (kv.page - 1)) >> 5),
                                           static_cast<int>(s0) & 31, static_cast<int>(s1) & 31};
        }
        if (lane == 0) s_n = n;
    }
    __syncthreads();
    const int n = s_n, D = kv.dim, oct = D / 8;
    const bool wide = kv.type != SV_KV_I8;
    for (int t = threadIdx.x; n && t < oct + D + 2; t += 256) {
        if (t < oct) {  // eight elements of the key
            if (wide) move_all<u32x4>(moves, n, [=](int k) { return (t * 32 + k) * 16; });
            else move_all<u32x2>(moves, n, [=](int k) { return (t * 32 + k) * 8; });
        } else if (t < oct + D) {  // one element of the value
            const int d = t - oct;
            if (wide) move_all<uint16_t>(moves, n, [=](int k) { return (32 * D + ((k >> 3) * D + d) * 8 + (k & 7)) * 2; });
            else move_all<uint8_t>(moves, n, [=](int k) { return 32 * D + ((k >> 3) * D + d) * 8 + (k & 7); });
        } else if (!wide) {  // the scales of the key and the value
            const int h = t - oct - D;
            move_all<uint32_t>(moves, n, [=](int k) { return 64 * D + (32 * h + k) * 4; });
        }
    }
}

__global__ __launch_bounds__(kBookThreads) void kv_fork_kernel(KvDev kv, const int32_t *src, const int32_t *dst,
                                                               int n) {
    fetch_args<sizeof(KvDev) + 24>();
    __shared__ int cnt[SV_KV_MAX_SEQS];
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid == 0) bad = 0;
    __syncthreads();
    for (int i = wave; i < n; i += kBookWaves) {
        const int s = gld(src + i), d = gld(dst + i);
        bool wrong = s < 0 || s >= kv.seqs || d < 0 || d >= kv.seqs;
        for (int at = 0; at < n && !wrong; at += 64) {
            const int j = at + lane;
            wrong = __any(j < n && ((j < i && gld(dst + j) == d) || gld(src + j) == d));
        }
        if (!wrong) wrong = gld(kv.len + d) != 0 || gld(kv.table + static_cast<int64_t>(d) * kv.width) >= 0;
        if (lane == 0) {
            int part = 0;
            if (wrong) {
                bad = 1;
            } else {
                const int64_t len = kv_len_of(kv, s);
                part = (len & (kv.page - 1)) && kv_page_of(kv, s, len >> kv.page_shift) >= 0;
            }
            cnt[i] = part;
        }
    }
    __syncthreads();
    const int total = scan_counts(cnt, n);
    const int fc = min(max(gld(kv.ctl), 0), kv.n_pages);
    if (bad || total > fc) {
        if (tid == 0) {
            kv_flag(kv, bad ? SV_KV_BAD_FORK : SV_KV_NO_PAGES);
            gst(kv.ctl + 2, 0);
        }
        return;
    }
    for (int i = wave; i < n; i += kBookWaves) {
        const int s = gld(src + i), d = gld(dst + i);
        const int64_t len = kv_len_of(kv, s), full = len >> kv.page_shift;
        for (int64_t e = lane; e < full; e += 64) {
            const int page = kv_page_of(kv, s, e);
            gst(kv.table + static_cast<int64_t>(d) * kv.width + e, page);
            if (page >= 0) add_dev(kv.refs + page, 1);
        }
        if (lane == 0) {
            const int part = (len & (kv.page - 1)) && kv_page_of(kv, s, full) >= 0;
            if (part) {
                const int page = gld(kv.free_ids + (fc - 1 - cnt[i]));
                if (page >= 0 && page < kv.n_pages) {
                    gst(kv.table + static_cast<int64_t>(d) * kv.width + full, page);
                    gst(kv.refs + page, 1);
                }
            }
            gst(kv.len + d, static_cast<int32_t>(len));
        }
    }
    __syncthreads();
    if (tid == 0) {
        gst(kv.ctl, fc - total);
        gst(kv.ctl + 2, n);
    }
}

// 16-byte pieces by a workgroup of 256, N a thread on their way at once,
// written past the caches; ONCE: nothing else reads them either.
template <int N, bool ONCE>
__device__ __forceinline__ void copy_pieces(uint8_t *to, const uint8_t *from, int n) {
    const SV_GLOBAL u32x4 *source = (const SV_GLOBAL u32x4 *)from;
    SV_GLOBAL u32x4 *target = (SV_GLOBAL u32x4 *)to;
    for (int t = threadIdx.x; t < n; t += 256 * N) {
        u32x4 x[N];
#pragma unroll
        for (int i = 0; i < N; i++)
            if (t + 256 * i < n) x[i] = ONCE ? __builtin_nontemporal_load(source + t + 256 * i) : source[t + 256 * i];
#pragma unroll
        for (int i = 0; i < N; i++)
            if (t + 256 * i < n) __builtin_nontemporal_store(x[i], target + t + 256 * i);
    }
}

// Copies the used blocks of the part-filled pages, one workgroup per (head
// and layer, pair): contiguous 16-byte pieces, bound by memory bandwidth.  142
// MB written and 9 MB read, again and again, in 31 us; 64 MB copied in 18 us
// (one piece a thread at a time and through the caches 36 and 22).
__global__ __launch_bounds__(256) void kv_fork_copy_kernel(KvDev kv, const int32_t *src, const int32_t *dst, int n) {
    fetch_args<sizeof(KvDev) + 24>();
    if (gld(kv.ctl + 2) != n) return;  // the bookkeeping refused the call
    const int i = blockIdx.y, head = blockIdx.x % kv.heads, layer = blockIdx.x / kv.heads;
    const int s = gld(src + i), d = gld(dst + i);
    const int64_t len = kv_len_of(kv, s);
    const int used = static_cast<int>((len & (kv.page - 1)) + kBlk - 1) >> 5;
    if (!used) return;
    const int p0 = kv_page_of(kv, s, len >> kv.page_shift), p1 = kv_page_of(kv, d, len >> kv.page_shift);
    if (p0 < 0 || p1 < 0) return;
    copy_pieces<8, false>(kv_block(kv, layer, p1, head, 0), kv_block(kv, layer, p0, head, 0),
                          used * static_cast<int>(kv.blk_bytes / 16));
}

// ------------------------------------------------------------- compaction
// Workspace: map[n_pages] (new id of a moved page), holes[n_pages],
// moves[n_pages] (its old id).
__global__ __launch_bounds__(kBookThreads) void kv_compact_kernel(KvDev kv, int32_t *map, int32_t *holes,
                                                                  int32_t *moves) {
    fetch_args<sizeof(KvDev) + 24>();
    __shared__ int cnt[kBookThreads];
    const int tid = threadIdx.x;
    const int fc = min(max(gld(kv.ctl), 0), kv.n_pages), live = kv.n_pages - fc;
    int n_holes = 0, n_moves = 0;
    for (int pass = 0; pass < 2; pass++) {
        const int lo = pass ? live : 0, hi = pass ? kv.n_pages : live;
        int run = 0;
        for (int at = lo; at < hi; at += kBookThreads) {
            const int id = at + tid;
            const bool held = id < hi && gld(kv.refs + id) > 0;
            const bool flag = id < hi && held == (pass == 1);
            cnt[tid] = flag;
            __syncthreads();
            const int total = scan_counts(cnt, kBookThreads);
            const int rank = run + cnt[tid];
            if (flag) st_dev((pass ? moves : holes) + rank, id);
            run += total;
            __syncthreads();
        }
        if (pass) n_moves = run;
        else n_holes = run;
    }
    drain();
    __syncthreads();
    // as many holes as moves, unless the caller's counts are wrong: then the
    // rest stays where it is
    for (int i = n_holes + tid; i < n_moves; i += kBookThreads) gst(map + ld_dev(moves + i), ld_dev(moves + i));
    if (n_moves > n_holes) n_moves = n_holes;
    for (int i = tid; i < n_moves; i += kBookThreads) {
        const int from = ld_dev(moves + i), to = ld_dev(holes + i);
        gst(map + from, to);
        gst(kv.refs + to, gld(kv.refs + from));
        gst(kv.refs + from, 0);
    }
    for (int i = tid; i < fc; i += kBookThreads) gst(kv.free_ids + i, kv.n_pages - 1 - i);
    if (tid == 0) gst(kv.ctl + 2, n_moves);
}

// The table's entries of moved pages, and the moves themselves in pieces of
// 16 KB: sources all lie above destinations, so pieces go in any order.
// Bound by memory bandwidth: 1.2 GB moved in 430 us, 5.6 TB/s read and
// written (through the caches 457, four pieces a thread at a time 437).
constexpr int kPiece = 16384;
__global__ __launch_bounds__(256) void kv_compact_move_kernel(KvDev kv, const int32_t *map, const int32_t *holes,
                                                              const int32_t *moves) {
    fetch_args<sizeof(KvDev) + 24>();
    const int n_moves = gld(kv.ctl + 2);
    const int fc = min(max(gld(kv.ctl), 0), kv.n_pages), live = kv.n_pages - fc;
    const int64_t entries = static_cast<int64_t>(kv.seqs) * kv.width;
    if (n_moves == 0) return;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < entries;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int page = gld(kv.table + i);
        if (page >= live && page < kv.n_pages) gst(kv.table + i, gld(map + page));
    }
    const int64_t pieces = (kv.page_bytes + kPiece - 1) / kPiece;
    const int64_t units = pieces * n_moves * kv.layers;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t piece = u % pieces, mv = u / pieces % n_moves, layer = u / pieces / n_moves;
        const uint8_t *from = kv.data + (layer * kv.n_pages + gld(moves + mv)) * kv.page_bytes + piece * kPiece;
        uint8_t *to = kv.data + (layer * kv.n_pages + gld(holes + mv)) * kv.page_bytes + piece * kPiece;
        const int64_t left = kv.page_bytes - piece * kPiece;
        const int n = static_cast<int>((left < kPiece ? left : kPiece) / 16);
        copy_pieces<1, true>(to, from, n);
    }
}

// ---------------------------------------------------------- rows in, out
// What one element of the cache's types is made of.
__device__ __forceinline__ uint16_t bits_f16(float x) {
    const _Float16 h = static_cast<_Float16>(x);
    uint16_t b;
    __builtin_memcpy(&b, &h, 2);
    return b;
}
__device__ __forceinline__ uint16_t bits_bf16(float x) {
    const __bf16 h = static_cast<__bf16>(x);
    uint16_t b;
    __builtin_memcpy(&b, &h, 2);
    return b;
}
__device__ __forceinline__ float float_bf16(uint32_t b) { return __uint_as_float(b << 16); }

// The rotation of pair (x0, x1): products and sums rounded one by one, so
// the result does not depend on where it is taken.
__device__ __forceinline__ float rot_first(float x0, float x1, float c, float s) {
    return __fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s));
}
__device__ __forceinline__ float rot_second(float x0, float x1, float c, float s) {
    return __fadd_rn(__fmul_rn(x1, c), __fmul_rn(x0, s));
}

// Rows into the cache: a workgroup takes the 32 slots of one block of one
// head, stages the rows that fall into it in LDS (keys, then values), and
// writes the block's pieces from there: eight elements of a key, eight slots
// of a value, so that neighbouring lanes write neighbouring 16-byte pieces
// although the fp32 rows are read along the head dimension.  Bound by
// latency for the rows of a round, by memory bandwidth for a prompt: 5 rows of
// 8 heads of 128 take 5.6 us, 4 prompts of up to 3000 rows 30 us (keys and
// values by one workgroup, rotated in LDS: 8.5 and 38; the head dimension an
// argument: 5.8 and 32).
constexpr int kPad = 4;  // floats past a staged row, against bank conflicts
template <int TYPE, int D>
__global__ __launch_bounds__(256) void kv_append_kernel(KvDev kv, int layer, sv_kv_batch bt, const float *k,
                                                        const float *v, sv_kv_rope rope) {
    fetch_args<sizeof(KvDev) + sizeof(sv_kv_batch) + sizeof(sv_kv_rope) + 24>();
    extern __shared__ float rows[];  // [32][dim + kPad]
    __shared__ float scale[kBlk];
    __shared__ int s_sid;
    const int tid = threadIdx.x, b = blockIdx.y, what = blockIdx.z;  // keys, values
    const int head = blockIdx.x % kv.heads, nth = blockIdx.x / kv.heads;
    int sid = b;
    if (bt.seq) {
        if (tid < 64) {
            const int first = first_sid(bt.seq, b, kv.seqs);
            if (tid == 0) s_sid = first;
        }
        __syncthreads();
        sid = s_sid;
    }
    if (sid < 0 || sid >= kv.seqs) return;
    const int64_t len = kv_len_of(kv, sid);
    const int n = kv_rows_of(bt.n_new, b, bt.M);
    const int64_t blk = (len >> 5) + nth;                    // the block, counted from the sequence's start
    const int lo = static_cast<int>(max(len - blk * kBlk, int64_t(0)));            // its first and
    const int hi = static_cast<int>(min(len + n - blk * kBlk, int64_t(kBlk)));     // one past its last new slot
    if (lo >= hi) return;
    const int page = kv_page_of(kv, sid, blk >> kv.blk_shift);  // not waited for yet
    constexpr int ld = D + kPad, quads = D / 4;
    const float *x = what ? v : k;
    // rotated on the way, a quad at a time, where its pairs are whole
    const int rot = what ? 0 : rope.rot, half = rot / 2;
    const bool turned = !what && rope.mode != SV_ROPE_NONE, by_quads = turned && rot % 8 == 0;
    auto position = [&](int m) {
        int64_t pos = len + m;
        if (bt.tree) pos = len + __popc(gld(bt.tree + static_cast<int64_t>(b) * bt.M + m) & ((1u << m) - 1));
        return min(pos, static_cast<int64_t>(rope.n_pos) - 1);
    };
    for (int i = tid; i < (hi - lo) * quads; i += 256) {
        const int s = lo + i / quads, d = i % quads * 4;
        const int m = static_cast<int>(blk * kBlk + s - len);
        const float *row = x + ((static_cast<int64_t>(b) * bt.M + m) * kv.heads + head) * D;
        u32x4 raw = gld(reinterpret_cast<const u32x4 *>(row + d));
        if (by_quads && d < rot) {
            const float *cs = rope.table + position(m) * rot;
            const float y[4] = {__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z), __uint_as_float(raw.w)};
            float z[4];
            if (rope.mode == SV_ROPE_PAIRS) {
                const u32x4 w = gld(reinterpret_cast<const u32x4 *>(cs + d));
                z[0] = rot_first(y[0], y[1], __uint_as_float(w.x), __uint_as_float(w.y));
                z[1] = rot_second(y[0], y[1], __uint_as_float(w.x), __uint_as_float(w.y));
                z[2] = rot_first(y[2], y[3], __uint_as_float(w.z), __uint_as_float(w.w));
                z[3] = rot_second(y[2], y[3], __uint_as_float(w.z), __uint_as_float(w.w));
            } else {
                const bool second = d >= half;
                const int p = second ? d - half : d;
                const u32x4 mate = gld(reinterpret_cast<const u32x4 *>(row + (second ? p : p + half)));
                const u32x4 w0 = gld(reinterpret_cast<const u32x4 *>(cs + 2 * p)), w1 = gld(reinterpret_cast<const u32x4 *>(cs + 2 * p + 4));
                const uint32_t c4[4] = {w0.x, w0.z, w1.x, w1.z}, s4[4] = {w0.y, w0.w, w1.y, w1.w};
                const uint32_t t4[4] = {mate.x, mate.y, mate.z, mate.w};
                for (int e = 0; e < 4; e++) {
                    const float t = __uint_as_float(t4[e]), co = __uint_as_float(c4[e]), si = __uint_as_float(s4[e]);
                    z[e] = second ? rot_second(t, y[e], co, si) : rot_first(y[e], t, co, si);
                }
            }
            raw = u32x4{__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3])};
        }
        *reinterpret_cast<u32x4 *>(rows + s * ld + d) = raw;
    }
    if (page < 0) {
        if (tid == 0) kv_flag(kv, SV_KV_NO_SLOT);
        return;
    }
    uint8_t *to = kv_block(kv, layer, page, head, static_cast<int>(blk & ((1 << kv.blk_shift) - 1)));
    __syncthreads();
    if (turned && !by_quads) {
        for (int i = tid; i < (hi - lo) * half; i += 256) {
            const int s = lo + i / half, c = i % half;
            const float *cs = rope.table + (position(static_cast<int>(blk * kBlk + s - len)) * half + c) * 2;
            const float co = gld(cs), si = gld(cs + 1);
            float *p0 = rows + s * ld + (rope.mode == SV_ROPE_PAIRS ? 2 * c : c);
            float *p1 = rope.mode == SV_ROPE_PAIRS ? p0 + 1 : p0 + half;
            const float x0 = *p0, x1 = *p1;
            *p0 = rot_first(x0, x1, co, si);
            *p1 = rot_second(x0, x1, co, si);
        }
        __syncthreads();
    }
    if (TYPE == SV_KV_I8) {
        // eight lanes a row: the largest magnitude, and whether all are finite
        const int s = tid >> 3;
        float a = 0.0f;
        bool fine = true;
        if (s >= lo && s < hi) {
            for (int c = tid & 7; c < D; c += 8) {
                const float y = fabsf(rows[s * ld + c]);
                fine &= y <= 3.4028234664e38f;
                a = fmaxf(a, y);
            }
        }
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) {
            a = fmaxf(a, __shfl_xor(a, o, 8));
            const int other = __shfl_xor(static_cast<int>(fine), o, 8);  // by every lane, whatever its own answer
            fine &= other != 0;
        }
        if ((tid & 7) == 0 && s >= lo && s < hi) {
            const float d = a / 127.0f;
            const float w = fine ? (d >= 1.17549435e-38f ? d : 0.0f) : __uint_as_float(0x7FC00000u);
            scale[s] = w;
            gst(reinterpret_cast<float *>(to + 64 * D) + 32 * what + s, w);
        }
        __syncthreads();
    }
    if (!what) {
        for (int i = tid; i < 32 * (D / 8); i += 256) {
            const int s = i & 31, o = i >> 5;
            if (s < lo || s >= hi) continue;
            const float *r = rows + s * ld + 8 * o;
            if (TYPE == SV_KV_I8) {
                const float w = scale[s], id = w > 0.0f ? 1.0f / w : 0.0f;
                uint32_t c[8];
                for (int e = 0; e < 8; e++) {
                    const float y = w > 0.0f ? fminf(fmaxf(roundf(r[e] * id), -127.0f), 127.0f) : 0.0f;
                    c[e] = static_cast<uint32_t>(static_cast<int>(y)) & 0xFFu;
                }
                u32x2 z;
                z.x = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
                z.y = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
                gst(reinterpret_cast<u32x2 *>(to) + i, z);
            } else {
                uint32_t c[8];
                for (int e = 0; e < 8; e++) c[e] = TYPE == SV_KV_F16 ? bits_f16(r[e]) : bits_bf16(r[e]);
                u32x4 z;
                z.x = c[0] | c[1] << 16;
                z.y = c[2] | c[3] << 16;
                z.z = c[4] | c[5] << 16;
                z.w = c[6] | c[7] << 16;
                gst(reinterpret_cast<u32x4 *>(to) + i, z);
            }
        }
    } else {
        for (int i = tid; i < 4 * D; i += 256) {
            const int d = i % D, s0 = i / D * 8;
            if (s0 + 8 <= lo || s0 >= hi) continue;
            uint32_t c[8];
            for (int e = 0; e < 8; e++) {
                const int s = s0 + e;
                c[e] = 0;
                if (s < lo || s >= hi) continue;
                const float y = rows[s * ld + d];
                if (TYPE == SV_KV_I8) {
                    const float w = scale[s], id = w > 0.0f ? 1.0f / w : 0.0f;
                    const float z = w > 0.0f ? fminf(fmaxf(roundf(y * id), -127.0f), 127.0f) : 0.0f;
                    c[e] = static_cast<uint32_t>(static_cast<int>(z)) & 0xFFu;
                } else {
                    c[e] = TYPE == SV_KV_F16 ? bits_f16(y) : bits_bf16(y);
                }
            }
            const bool all = s0 >= lo && s0 + 8 <= hi;
            if (TYPE == SV_KV_I8) {
                uint8_t *z = to + 32 * D + i * 8;
                if (all) {
                    u32x2 w;
                    w.x = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
                    w.y = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
                    gst(reinterpret_cast<u32x2 *>(z), w);
                } else {
                    for (int e = 0; e < 8; e++)
                        if (s0 + e >= lo && s0 + e < hi) gst(z + e, static_cast<uint8_t>(c[e]));
                }
            } else {
                uint16_t *z = reinterpret_cast<uint16_t *>(to + 64 * D) + i * 8;
                if (all) {
                    u32x4 w;
                    w.x = c[0] | c[1] << 16;
                    w.y = c[2] | c[3] << 16;
                    w.z = c[4] | c[5] << 16;
                    w.w = c[6] | c[7] << 16;
                    gst(reinterpret_cast<u32x4 *>(z), w);
                } else {
                    for (int e = 0; e < 8; e++)
                        if (s0 + e >= lo && s0 + e < hi) gst(z + e, static_cast<uint16_t>(c[e]));
                }
            }
        }
    }
}

// Rows out of the cache: a workgroup per block of 32 slots and head, as
// above: pieces of the block to LDS, rows from LDS to fp32.  5 rows of 8
// heads 4 us, 8124 rows of 8 heads 18 us.
template <int TYPE, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(KvDev kv, int layer, sv_kv_batch bt, const int32_t *start,
                                                      float *k_out, float *v_out) {
    fetch_args<sizeof(KvDev) + sizeof(sv_kv_batch) + 32>();
    extern __shared__ float rows[];  // [32][dim + kPad]
    const int tid = threadIdx.x, b = blockIdx.y, what = k_out ? blockIdx.z : 1;  // keys, values
    const int head = blockIdx.x % kv.heads, nth = blockIdx.x / kv.heads;
    const int sid = bt.seq ? gld(bt.seq + b) : b;
    if (sid < 0 || sid >= kv.seqs) return;
    const int64_t first = start ? static_cast<int64_t>(gld(start + b)) : kv_len_of(kv, sid);
    const int n = kv_rows_of(bt.n_new, b, bt.M);
    const int64_t blk = (first >> 5) + nth;
    const int lo = static_cast<int>(max(first - blk * kBlk, int64_t(0)));
    const int hi = static_cast<int>(min(first + n - blk * kBlk, int64_t(kBlk)));
    if (lo >= hi) return;
    const int page = blk < 0 ? -1 : kv_page_of(kv, sid, blk >> kv.blk_shift);
    const uint8_t *from =
        page < 0 ? nullptr : kv_block(kv, layer, page, head, static_cast<int>(blk & ((1 << kv.blk_shift) - 1)));
    constexpr int ld = D + kPad, quads = D / 4;
    float *out = what ? v_out : k_out;
    if (from) {
        for (int i = tid; i < 4 * D; i += 256) {  // 32 (D / 8) pieces of the key, 4 D of the value: as many
            const int s = what ? i / D * 8 : i & 31, d = what ? i % D : (i >> 5) * 8;
            if (what ? s + 8 <= lo || s >= hi : s < lo || s >= hi) continue;
            float x[8];
            if (TYPE == SV_KV_I8) {
                const uint2 c = gld8(from + (what ? 32 * D : 0) + i * 8);
                const float *sc = reinterpret_cast<const float *>(from + 64 * D) + 32 * what;
                for (int e = 0; e < 8; e++) {
                    const int code = static_cast<int8_t>((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
                    x[e] = static_cast<float>(code) * gld(sc + (what ? s + e : s));
                }
            } else {
                const uint4 c = gld16(from + (what ? 64 * D : 0) + i * 16);
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
                for (int e = 0; e < 8; e++) {
                    const uint32_t h = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                    x[e] = TYPE == SV_KV_F16 ? half_bits_to_float(h) : float_bf16(h);
                }
            }
            for (int e = 0; e < 8; e++) {
                if (what) rows[(s + e) * ld + d] = x[e];
                else rows[s * ld + d + e] = x[e];
            }
        }
    } else {
        for (int i = tid; i < 32 * D; i += 256) rows[i / D * ld + i % D] = 0.0f;
    }
    __syncthreads();
    for (int i = tid; i < (hi - lo) * quads; i += 256) {
        const int s = lo + i / quads, c = i % quads;
        const int64_t m = blk * kBlk + s - first;
        const float4 x = *reinterpret_cast<const float4 *>(rows + s * ld + 4 * c);
        u32x4 z = {__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z), __float_as_uint(x.w)};
        gst(reinterpret_cast<u32x4 *>(out + ((static_cast<int64_t>(b) * bt.M + m) * kv.heads + head) * D + 4 * c), z);
    }
}

// The kernels of a cache's type and head dimension.
using AppendFn = void (*)(KvDev, int, sv_kv_batch, const float *, const float *, sv_kv_rope);
using ReadFn = void (*)(KvDev, int, sv_kv_batch, const int32_t *, float *, float *);
struct RowFns {
    AppendFn append;
    ReadFn read;
};
template <int TYPE>
static RowFns row_fns_of(int dim) {
    static constexpr RowFns fns[] = {
        {kv_append_kernel<TYPE, 32>, kv_read_kernel<TYPE, 32>},   {kv_append_kernel<TYPE, 64>, kv_read_kernel<TYPE, 64>},
        {kv_append_kernel<TYPE, 96>, kv_read_kernel<TYPE, 96>},   {kv_append_kernel<TYPE, 128>, kv_read_kernel<TYPE, 128>},
        {kv_append_kernel<TYPE, 160>, kv_read_kernel<TYPE, 160>}, {kv_append_kernel<TYPE, 192>, kv_read_kernel<TYPE, 192>},
        {kv_append_kernel<TYPE, 224>, kv_read_kernel<TYPE, 224>}, {kv_append_kernel<TYPE, 256>, kv_read_kernel<TYPE, 256>}};
    static_assert(sizeof(fns) / sizeof(fns[0]) == kMaxDim / 32, "a kernel for every head dimension");
    return fns[dim / 32 - 1];
}
static RowFns row_fns(const KvDev &d) {
    return d.type == SV_KV_F16    ? row_fns_of<SV_KV_F16>(d.dim)
           : d.type == SV_KV_BF16 ? row_fns_of<SV_KV_BF16>(d.dim)
                                  : row_fns_of<SV_KV_I8>(d.dim);
}

// Blocks of 32 slots that M rows can touch, from any slot on.
static int64_t row_blocks(int M) { return (static_cast<int64_t>(M) + 30) / 32 + 1; }

}  // namespace sv

using namespace sv;

extern "C" size_t sv_kv_page_bytes(int32_t type, int32_t heads, int32_t dim, int32_t page) {
    if (!kv_shape_ok(type, heads, dim, page)) return 0;
    return static_cast<size_t>(heads) * (page / kBlk) * kv_block_bytes(type, dim);
}

extern "C" size_t sv_kv_data_bytes(const sv_kv *kv) {
    if (!kv || kv->layers < 1 || kv->layers > kKvMaxLayers || kv->n_pages < 1 || kv->n_pages > kKvMaxPages) return 0;
    const size_t page = sv_kv_page_bytes(kv->type, kv->heads, kv->dim, kv->page);
    const size_t pages = static_cast<size_t>(kv->layers) * kv->n_pages;  // at most 2^36
    if (!page || static_cast<int64_t>(kv->layers) * kv->heads >= (1 << 23) || pages >= kKvMaxBytes / page) return 0;
    return pages * page;
}

extern "C" int sv_kv_init(const sv_kv *kv, void *stream) {
    KvDev d;
    const int rc = kv_check(kv, "kv_init", &d);
    if (rc) return rc;
    hipLaunchKernelGGL(kv_init_kernel, dim3(64), dim3(kBookThreads), 0, as_stream(stream), d);
    return hip_check(hipGetLastError(), "kv_init launch");
}

// Rows of a reservation: as long as a table row, and no longer than a prompt
// that append takes.
constexpr int kMaxRows = 1 << 24;

extern "C" int sv_kv_reserve(const sv_kv *kv, const sv_kv_batch *batch, void *stream) {
    KvDev d;
    int rc = kv_check(kv, "kv_reserve", &d);
    if (rc) return rc;
    sv_kv_batch bt = batch ? *batch : sv_kv_batch{};
    bt.tree = nullptr;
    rc = kv_check_batch(d, batch ? &bt : nullptr, "kv_reserve", kMaxRows);
    if (rc) return rc;
    hipLaunchKernelGGL(kv_reserve_kernel, dim3(1), dim3(kBookThreads), 0, as_stream(stream), d, bt);
    return hip_check(hipGetLastError(), "kv_reserve launch");
}

extern "C" int sv_kv_append(const sv_kv *kv, int32_t layer, const sv_kv_batch *batch, const float *k, const float *v,
                            const sv_kv_rope *rope, void *stream) {
    KvDev d;
    int rc = kv_check(kv, "kv_append", &d);
    if (!rc) rc = kv_check_batch(d, batch, "kv_append", kMaxRows);
    if (!rc) rc = kv_check_rope(d, rope, "kv_append");
    if (rc) return rc;
    SV_REQUIRE(layer >= 0 && layer < d.layers, SV_ERR_ARG, "kv_append: layer out of range");
    SV_REQUIRE(k && v, SV_ERR_ARG, "kv_append: NULL buffer");
    SV_REQUIRE(aligned(k, 16) && aligned(v, 16), SV_ERR_ALIGN, "kv_append: k and v must be 16-byte aligned");
    const int64_t gx = row_blocks(batch->M) * d.heads;
    SV_REQUIRE(gx < (1ll << 24), SV_ERR_SHAPE, "kv_append: too large");
    const sv_kv_rope r = rope ? *rope : sv_kv_rope{};
    const size_t lds = kBlk * (d.dim + kPad) * sizeof(float);
    const dim3 grid(static_cast<unsigned>(gx), batch->B, 2);
    hipLaunchKernelGGL(row_fns(d).append, grid, dim3(256), lds, as_stream(stream), d, layer, *batch, k, v, r);
    return hip_check(hipGetLastError(), "kv_append launch");
}

extern "C" int sv_kv_read(const sv_kv *kv, int32_t layer, const sv_kv_batch *batch, const int32_t *start,
                          float *k_out, float *v_out, void *stream) {
    KvDev d;
    int rc = kv_check(kv, "kv_read", &d);
    if (rc) return rc;
    sv_kv_batch bt = batch ? *batch : sv_kv_batch{};
    bt.tree = nullptr;
    rc = kv_check_batch(d, batch ? &bt : nullptr, "kv_read", kMaxRows);
    if (rc) return rc;
    SV_REQUIRE(layer >= 0 && layer < d.layers, SV_ERR_ARG, "kv_read: layer out of range");
    SV_REQUIRE(k_out || v_out, SV_ERR_ARG, "kv_read: NULL buffer");
    SV_REQUIRE((!k_out || aligned(k_out, 16)) && (!v_out || aligned(v_out, 16)) && (!start || aligned(start, 4)),
               SV_ERR_ALIGN, "kv_read: outputs must be 16-byte aligned, start 4-byte aligned");
    const int64_t gx = row_blocks(bt.M) * d.heads;
    SV_REQUIRE(gx < (1ll << 24), SV_ERR_SHAPE, "kv_read: too large");
    const size_t lds = kBlk * (d.dim + kPad) * sizeof(float);
    hipLaunchKernelGGL(row_fns(d).read, dim3(static_cast<unsigned>(gx), bt.B, k_out && v_out ? 2 : 1), dim3(256), lds,
                       as_stream(stream), d, layer, bt, start, k_out, v_out);
    return hip_check(hipGetLastError(), "kv_read launch");
}

extern "C" int sv_kv_commit(const sv_kv *kv, const sv_kv_batch *batch, const int32_t *accepted, int32_t stride,
                            const int32_t *path, void *stream) {
    KvDev d;
    int rc = kv_check(kv, "kv_commit", &d);
    if (rc) return rc;
    sv_kv_batch bt = batch ? *batch : sv_kv_batch{};
    bt.tree = nullptr;
    rc = kv_check_batch(d, batch ? &bt : nullptr, "kv_commit", kMaxRows);
    if (rc) return rc;
    SV_REQUIRE(accepted && stride >= 1, SV_ERR_ARG, "kv_commit: accepted must not be NULL and stride at least 1");
    SV_REQUIRE(!path || bt.M <= 32, SV_ERR_ARG, "kv_commit: a path needs M <= 32");
    SV_REQUIRE(static_cast<int64_t>(bt.B) * d.width < (1ll << 31), SV_ERR_SHAPE, "kv_commit: B * width must be below 2^31");
    SV_REQUIRE(aligned(accepted, 4) && (!path || aligned(path, 4)), SV_ERR_ALIGN,
               "kv_commit: int32 buffers must be 4-byte aligned");
    if (path)
        hipLaunchKernelGGL(kv_commit_move_kernel, dim3(d.heads * d.layers, bt.B), dim3(256), 0, as_stream(stream), d,
                           bt, accepted, stride, path);
    hipLaunchKernelGGL(kv_commit_kernel, dim3(1), dim3(kBookThreads), 0, as_stream(stream), d, bt, accepted, stride,
                       path);
    return hip_check(hipGetLastError(), "kv_commit launch");
}

extern "C" int sv_kv_fork(const sv_kv *kv, const int32_t *src, const int32_t *dst, int32_t n, void *stream) {
    KvDev d;
    const int rc = kv_check(kv, "kv_fork", &d);
    if (rc) return rc;
    SV_REQUIRE(src && dst, SV_ERR_ARG, "kv_fork: NULL buffer");
    SV_REQUIRE(n >= 1 && n <= SV_KV_MAX_SEQS, SV_ERR_ARG, "kv_fork: n must be in [1, 4096]");
    SV_REQUIRE(aligned(src, 4) && aligned(dst, 4), SV_ERR_ALIGN, "kv_fork: int32 buffers must be 4-byte aligned");
    hipLaunchKernelGGL(kv_fork_kernel, dim3(1), dim3(kBookThreads), 0, as_stream(stream), d, src, dst, n);
    hipLaunchKernelGGL(kv_fork_copy_kernel, dim3(d.heads * d.layers, n), dim3(256), 0, as_stream(stream), d, src, dst,
                       n);
    return hip_check(hipGetLastError(), "kv_fork launch");
}

extern "C" int sv_kv_release(const sv_kv *kv, const int32_t *ids, int32_t n, void *stream) {
    KvDev d;
    const int rc = kv_check(kv, "kv_release", &d);
    if (rc) return rc;
    SV_REQUIRE(ids, SV_ERR_ARG, "kv_release: NULL buffer");
    SV_REQUIRE(n >= 1 && n <= SV_KV_MAX_SEQS, SV_ERR_ARG, "kv_release: n must be in [1, 4096]");
    SV_REQUIRE(static_cast<int64_t>(n) * d.width < (1ll << 31), SV_ERR_SHAPE, "kv_release: n * width must be below 2^31");
    SV_REQUIRE(aligned(ids, 4), SV_ERR_ALIGN, "kv_release: int32 buffers must be 4-byte aligned");
    hipLaunchKernelGGL(kv_release_kernel, dim3(1), dim3(kBookThreads), 0, as_stream(stream), d, ids, n);
    return hip_check(hipGetLastError(), "kv_release launch");
}

extern "C" size_t sv_kv_compact_workspace_bytes(const sv_kv *kv) {
    if (!kv || kv->n_pages < 1 || kv->n_pages > kKvMaxPages) return 0;
    return static_cast<size_t>(kv->n_pages) * 12;
}

extern "C" int sv_kv_compact(const sv_kv *kv, void *workspace, size_t ws_bytes, void *stream) {
    KvDev d;
    const int rc = kv_check(kv, "kv_compact", &d);
    if (rc) return rc;
    const size_t need = sv_kv_compact_workspace_bytes(kv);
    SV_REQUIRE(workspace && ws_bytes >= need, SV_ERR_WORKSPACE,
               "kv_compact: workspace needs " + std::to_string(need) + " bytes");
    SV_REQUIRE(aligned(workspace, 4), SV_ERR_ALIGN, "kv_compact: the workspace must be 4-byte aligned");
    int32_t *map = static_cast<int32_t *>(workspace), *holes = map + d.n_pages, *moves = holes + d.n_pages;
    hipLaunchKernelGGL(kv_compact_kernel, dim3(1), dim3(kBookThreads), 0, as_stream(stream), d, map, holes, moves);
    hipLaunchKernelGGL(kv_compact_move_kernel, dim3(2048), dim3(256), 0, as_stream(stream), d, map, holes, moves);
    return hip_check(hipGetLastError(), "kv_compact launch");
}

extern "C" int sv_kv_status(const sv_kv *kv, uint32_t *status) {
    KvDev d;
    int rc = kv_check(kv, "kv_status", &d);
    if (rc) return rc;
    SV_REQUIRE(status, SV_ERR_ARG, "kv_status: NULL status");
    rc = hip_check(hipDeviceSynchronize(), "kv_status: synchronise");
    if (rc) return rc;
    rc = hip_check(hipMemcpy(status, kv->ctl + 1, 4, hipMemcpyDeviceToHost), "kv_status: read");
    if (rc) return rc;
    const uint32_t zero = 0;
    return hip_check(hipMemcpy(kv->ctl + 1, &zero, 4, hipMemcpyHostToDevice), "kv_status: clear");
}
