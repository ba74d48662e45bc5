// kv_internal.h - layout and argument checks of the key-value cache, shared
// by its page operators (kv.hip) and its attention (kv_attn.hip).
#pragma once

#include "sv_internal.h"

namespace sv {

constexpr int kBlk = 32;             // slots of a block
constexpr int kMaxDim = 256;
constexpr int kKvMaxPages = 1 << 24;
constexpr int kKvMaxLayers = 4096, kKvMaxHeads = 4096;
constexpr size_t kKvMaxBytes = size_t(1) << 48;  // of a pool: offsets and sizes stay exact

// Bytes of one block (32 slots of one head).
__host__ __device__ inline uint32_t kv_block_bytes(int type, int dim) {
    return type == SV_KV_I8 ? 64u * dim + 256u : 128u * dim;
}

// Argument block of the device code: the caller's descriptor with its
// derived sizes.
struct KvDev {
    uint8_t *data;
    int32_t *table, *len, *refs, *free_ids, *ctl;
    int32_t type, layers, heads, dim, n_pages, seqs, width;
    int32_t page;       // slots
    int32_t page_shift; // log2(page)
    int32_t blk_shift;  // log2(page / 32)
    uint32_t blk_bytes;
    int64_t page_bytes;
};

// Checks a cache descriptor (every buffer of it) and fills the device form.
int kv_check(const sv_kv *kv, const char *who, KvDev *out);
// Checks the sequences and rows of a call.
int kv_check_batch(const KvDev &kv, const sv_kv_batch *b, const char *who, int max_m);
int kv_check_rope(const KvDev &kv, const sv_kv_rope *r, const char *who);

// Requests all BYTES of a kernel's arguments at its start, line by line but
// together: a kernel begins with none of them in the scalar cache, and fields
// first used one after another would each wait for their own line.
template <int BYTES>
__device__ __forceinline__ void fetch_args() {
    typedef const __attribute__((address_space(4))) uint32_t *Args;
    const Args at = (Args)__builtin_amdgcn_kernarg_segment_ptr();
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < BYTES; i += 64) all |= at[i / 4];
    asm volatile("" ::"s"(all));
}

// The page of an entry, or -1 where the row has none.
__device__ __forceinline__ int kv_page_of(const KvDev &kv, int sid, int64_t entry) {
    if (entry < 0 || entry >= kv.width) return -1;
    const int p = gld(kv.table + static_cast<int64_t>(sid) * kv.width + entry);
    return p >= 0 && p < kv.n_pages ? p : -1;
}

// Start of block `blk` of a page, one layer and head.
__device__ __forceinline__ uint8_t *kv_block(const KvDev &kv, int layer, int page, int head, int blk) {
    return kv.data + (static_cast<int64_t>(layer) * kv.n_pages + page) * kv.page_bytes +
           (static_cast<int64_t>(head) << kv.blk_shift) * kv.blk_bytes + static_cast<int64_t>(blk) * kv.blk_bytes;
}

// A sequence's committed length, held within its table row.
__device__ __forceinline__ int64_t kv_len_of(const KvDev &kv, int sid) {
    const int64_t n = gld(kv.len + sid), cap = static_cast<int64_t>(kv.width) * kv.page;
    return n < 0 ? 0 : (n > cap ? cap : n);
}

__device__ __forceinline__ int kv_rows_of(const int32_t *n_new, int b, int M) {
    if (!n_new) return M;
    const int n = gld(n_new + b);
    return n < 0 ? 0 : (n > M ? M : n);
}

__device__ __forceinline__ void kv_flag(const KvDev &kv, uint32_t bits) {
    or_dev(reinterpret_cast<uint32_t *>(kv.ctl) + 1, bits);
}

}  // namespace sv
