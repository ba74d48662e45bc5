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
// Sums of kept weights are whole numbers: each weight, formed in fp64, counts
// as the nearest multiple of 2^-s with s = 63 - ceil(log2 V), at most 51
// (2^-45 for 151936 tokens), so a sum of V of them fits 64 bits and is the
// same in any order: atomics and any split of a row give the same bits.  A
// weight below half a step is never drawn: all of them together are less than
// V^2 2^-64 of the row (1e-9 for 151936).  Sums over a whole row that nothing
// filters are fp64, in the order of its chunks.
//
// One pass over the logits decides nearly every row:
//   scan    a workgroup per chunk of a row: a sample of the row gives a
//           threshold that about a thousand of its values pass; these are
//           listed in the order of their indices, with the chunk's largest
//           value and, if no top-k bounds what is kept, its sum of weights
//           (relative to the sample's largest value: the row's is not known);
//   finish  a workgroup per row: where what is kept lies within the list, the
//           border, the sum and the token come from the list, held in
//           registers; a row without filters takes its token from the chunks'
//           sums and one chunk.
// Rows whose kept set goes past the list (a flat distribution) take two more
// passes, split over chunks as well:
//   bins    amounts (elements, or steps of weight) by the distance from the
//           largest value, 16 bins to a factor of 2, which gives the border's
//           bin;
//   gather  the elements of that bin are listed, the kept weights above it
//           summed per chunk;
//   settle  a workgroup per row, as finish.
// What is left (a top-k past the list with a top-p as well, a bin of more
// elements than a list holds) is done by a workgroup from the row itself, by
// radix selection on the bits of z.
#include <algorithm>

#include "sv_internal.h"

namespace sv {

typedef unsigned long long u64;
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));  // rows may begin anywhere

constexpr int kRow = 1024;               // threads of a row's workgroup
constexpr int kScan = 512;               // threads of a chunk's
constexpr int kQuads = 8;                // quads of a chunk that a thread holds
constexpr int kChunk = kScan * kQuads * 4;
constexpr int kPer = 4, kList = kRow * kPer;  // listed elements that a row's workgroup holds
constexpr int kBins = 1024;
constexpr int kDigits = 2048;
constexpr int kSlots = 256;              // rows that are under way at once
constexpr int kFlatGrid = 1024;          // workgroups of the passes over flat rows
constexpr int64_t kMaxVocab = 1 << 24;
constexpr int64_t kMaxRows = 65535;

// What a chunk's workgroup leaves.
struct ChunkRec {
    float top;      // largest value; NaN if one is not a number or +inf
    int32_t n;      // listed elements, or more than the list holds
    int32_t rest;   // finite elements that are not listed: some, or none
    float tau, ref; // of the row: threshold of the list, the sample's largest value
    int32_t pad;
    union {
        double sum;  // of all weights, relative to ref; < 0: not formed
        u64 steps;   // of the kept weights above the border's bin
    };
};

enum { kDone, kFailed, kByCount, kByMass, kNoBorder, kSlow };

// A row's border and sum: what the outputs are made of, and what is known of
// a row that is not done.
struct RowState {
    int32_t kind, token;
    float top;
    uint32_t key;    // kept: keys above this one,
    int32_t cut;     // and those equal to it with a smaller index
    int32_t bin;     // the border's
    u64 want, above; // amounts: to be kept, and of the bins above
    double scale;    // weight times this: probability
};

struct SampleArgs {
    const float *logits;
    int64_t ld;
    const sv_sampling *params;
    int32_t per_row;  // 0: one for all rows
    int32_t V;
    int32_t shift;    // weights in steps of 2^-shift
    int32_t row0, rows;
    int32_t chunks, cap;  // of a row; list entries of a chunk
    const double *u;
    int32_t *tokens;
    float *probs, *kept;
    RowState *state;  // [all rows]
    ChunkRec *recs;   // [slots][chunks]
    uint2 *lists;     // [slots][chunks][cap]: bits of z, index
    u64 *bins;        // [slots][kBins]
    int32_t *flat;    // number of flat rows, then their slots
};

__device__ __forceinline__ const float *row_of(const SampleArgs &a, int r) { return a.logits + static_cast<int64_t>(r) * a.ld; }

struct Settings {
    bool fine;
    int k;            // elements to keep at most
    double per;       // log2(e) / T
    double p, least;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs &a, int r) {
    const sv_sampling *at = a.params + (a.per_row ? r : 0);
    const sv_sampling p{gld(&at->temperature), gld(&at->top_k), gld(&at->top_p), gld(&at->min_p)};
    Settings s;
    s.fine = p.temperature >= 0.0f && p.temperature < INFINITY && p.top_k >= 0 && p.top_p > 0.0f && p.top_p <= 1.0f &&
             p.min_p >= 0.0f && p.min_p <= 1.0f;
    const bool greedy = p.temperature == 0.0f;
    s.k = greedy ? 1 : p.top_k == 0 || p.top_k > a.V ? a.V : p.top_k;
    s.per = greedy ? 1.0 : 1.44269504088896340736 / static_cast<double>(p.temperature);
    s.p = p.top_p;
    s.least = p.min_p;
    return s;
}

// 2^y for y <= 1000 or so (relative error about 2^-52; below 2^-1080: 0):
// y = n + f, |f| <= 1/2, and the power series of 2^f up to f^12, whose rest is
// below (ln 2 / 2)^13 / 13! = 2e-16.
__device__ __forceinline__ double exp2_of(double y) {
    y = fmax(y, -1100.0);
    const double n = rint(y), x = (y - n) * 0.69314718055994530942;
    double s = 1.0 / 479001600.0;
    s = fma(s, x, 1.0 / 39916800.0);
    s = fma(s, x, 1.0 / 3628800.0);
    s = fma(s, x, 1.0 / 362880.0);
    s = fma(s, x, 1.0 / 40320.0);
    s = fma(s, x, 1.0 / 5040.0);
    s = fma(s, x, 1.0 / 720.0);
    s = fma(s, x, 1.0 / 120.0);
    s = fma(s, x, 1.0 / 24.0);
    s = fma(s, x, 1.0 / 6.0);
    s = fma(s, x, 0.5);
    s = fma(s, x, 1.0);
    s = fma(s, x, 1.0);
    return ldexp(s, static_cast<int>(n));
}
__device__ __forceinline__ double weight_of(float z, float one, double per) {
    return exp2_of((static_cast<double>(z) - static_cast<double>(one)) * per);
}
// w in [0, 1] to the nearest multiple of 2^-shift: 2^(52 - shift) + w leaves
// the multiple in the low bits of its fraction.
__device__ __forceinline__ u64 steps_of(double w, int shift) {
    const double one = __longlong_as_double(static_cast<long long>(1023 + 52 - shift) << 52);
    return static_cast<u64>(__double_as_longlong(one + w)) & ((1ull << 52) - 1);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ float bin_scale(double per) { return static_cast<float>(fmin(16.0 * per, 1e30)); }
// Bin of a finite z, 16 to a factor of 2 in weight; the last one holds all
// that is further.
__device__ __forceinline__ int bin_of(float z, float top, float scale) {
    return static_cast<int>(fminf((top - z) * scale, static_cast<float>(kBins - 1)));
}

struct Border {
    uint32_t key;
    int32_t cut;
    __device__ bool keeps(uint32_t k, int j) const { return k > key || (k == key && j < cut); }
};
__device__ __forceinline__ Border no_border() { return Border{float_key(-INFINITY), 0}; }

// ------------------------------------------------- sums over a workgroup
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {  // sum of the lanes up to and with this one
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const T t = __shfl_up(v, o, 64);
        if (lane >= o) v += t;
    }
    return v;
}
// Sum over the threads before this one; *all is that over all.  `room` holds a
// value for each wave; it may be used again after the next barrier.
template <int THREADS, typename T>
__device__ __forceinline__ T block_scan(T *room, T v, T *all) {
    const int wave = threadIdx.x >> 6;
    const T upto = wave_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) room[wave] = upto;
    __syncthreads();
    T before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; w++) {
        if (w == wave) before = sum;
        sum += room[w];
    }
    *all = sum;
    return before + upto - v;
}

struct RowShared {
    union {
        u64 hist[kDigits];
        struct {
            float z[kList];
            int32_t j[kList];
        } list;
    };
    uint32_t count[kBins];
    union {
        u64 wave[kRow / 64];
        double wave_f[kRow / 64];
    };
    u64 above, amount;
    double base;
    uint32_t lo, hi;
    int32_t digit, at, last, flags;
    int32_t offsets[kRow + 1];
};

// --------------------------------------- a border among listed elements
// Thread t holds elements kPer t .. of a list that is in the order of the
// indices; `in` says which are eligible.  Border of the first `want` (of their
// amounts) of them in falling order; want <= the sum.
template <bool MASS>
__device__ Border border_of(RowShared &sh, const uint32_t (&key)[kPer], const int32_t (&j)[kPer], const bool (&in)[kPer],
                            const u64 (&amount)[kPer], u64 want) {
    const int tid = threadIdx.x;
    u64 above = 0;
    uint32_t lo = ~0u, hi = 0;
    __syncthreads();
    if (tid == 0) {
        sh.lo = ~0u;
        sh.hi = 0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; i++)
        if (in[i]) {
            lo = min(lo, key[i]);
            hi = max(hi, key[i]);
        }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        lo = min(lo, static_cast<uint32_t>(__shfl_xor(lo, o, 64)));
        hi = max(hi, static_cast<uint32_t>(__shfl_xor(hi, o, 64)));
    }
    if ((tid & 63) == 0) {
        atomicMin(&sh.lo, lo);
        atomicMax(&sh.hi, hi);
    }
    __syncthreads();
    lo = sh.lo;
    hi = sh.hi;
    for (;;) {
        const int bits = hi > lo ? 32 - __clz(hi - lo) : 0, low = bits > 10 ? bits - 10 : 0;
        __syncthreads();
        sh.hist[tid] = 0;
        sh.count[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (in[i] && key[i] >= lo && key[i] <= hi) {
                const int d = (key[i] - lo) >> low;
                atomicAdd(&sh.count[d], 1u);
                if (MASS) atomicAdd(&sh.hist[d], amount[i]);
            }
        __syncthreads();
        const int d = kBins - 1 - tid;
        const u64 h = MASS ? sh.hist[d] : sh.count[d];
        u64 all;
        const u64 before = above + block_scan<kRow>(sh.wave, h, &all);
        if (before < want && before + h >= want) {
            sh.digit = d;
            sh.above = before;
            sh.amount = h;
        }
        __syncthreads();
        lo += static_cast<uint32_t>(sh.digit) << low;
        hi = min(hi, lo + ((1u << low) - 1));
        above = sh.above;
        const int number = sh.count[sh.digit];
        // one element, or all of the digit's: nothing is left to be told apart
        if (low > 0 && (number == 1 || (!MASS && above + sh.amount == want))) return Border{lo, INT32_MAX};
        if (low > 0) continue;
        const u64 each = sh.amount / number, need = (want - above + each - 1) / each;
        if (need >= static_cast<u64>(number)) return Border{lo, INT32_MAX};
        // the first `need` of the equal ones
        u64 mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; i++) mine += in[i] && key[i] == lo;
        u64 upto = block_scan<kRow>(sh.wave, mine, &all);
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (in[i] && key[i] == lo && ++upto == need) sh.at = j[i] + 1;
        __syncthreads();
        return Border{lo, sh.at};
    }
}

// -------------------------------------- a border from the row, bit by bit
// Moves the border so that the first `want` (of falling order) of what it
// keeps remain: of `want` elements, or of steps of weight.
template <bool MASS>
__device__ void select(const SampleArgs &a, RowShared &sh, const float *row, float top, double per, u64 want,
                       Border *border) {
    const int tid = threadIdx.x;
    const Border from = *border;
    uint32_t prefix = 0, known = 0;  // the bits of the key found so far, and which they are
    u64 above = 0;                   // amount above them
    for (int level = 0; level < 3; level++) {
        const int low = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        __syncthreads();
        for (int i = tid; i < kDigits; i += kRow) sh.hist[i] = 0;
        __syncthreads();
        for (int j = tid; j < a.V; j += kRow) {
            const float z = gld(row + j);
            const uint32_t k = float_key(z);
            if ((k & known) != prefix || !from.keeps(k, j)) continue;
            const u64 n = MASS ? steps_of(weight_of(z, top, per), a.shift) : 1;
            atomicAdd(&sh.hist[(k >> low) & ((1u << bits) - 1)], n);
        }
        __syncthreads();
        // digits in falling order, two a thread
        const int d1 = kDigits - 1 - 2 * tid, d0 = d1 - 1;
        const u64 h1 = sh.hist[d1], h0 = sh.hist[d0];
        u64 all;
        const u64 before = above + block_scan<kRow>(sh.wave, h1 + h0, &all);
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
    }
    // of the elements equal to the border the first `need`
    const u64 each = MASS ? steps_of(weight_of(value_of(prefix), top, per), a.shift) : 1;
    const u64 need = (want - above + each - 1) / each;
    u64 passed = 0;
    int cut = a.V;
    for (int j0 = 0; j0 < a.V; j0 += kRow) {
        const int j = j0 + tid;
        bool is = false;
        if (j < a.V) {
            const uint32_t k = float_key(gld(row + j));
            is = k == prefix && from.keeps(k, j);
        }
        u64 all;
        const u64 before = passed + block_scan<kRow>(sh.wave, static_cast<u64>(is), &all);
        if (is && before + 1 == need) sh.at = j + 1;
        passed += all;
        if (passed >= need) {
            __syncthreads();
            cut = sh.at;
            break;
        }
    }
    __syncthreads();
    *border = Border{prefix, cut};
}

// ------------------------------------------------------------- the token
// Steps past which the running sum has to go.
__device__ __forceinline__ u64 threshold(double u, u64 total) {
    const u64 t = static_cast<u64>(u * static_cast<double>(total));
    return t < total ? t : total - 1;
}
// The first element of [j0, j1) at which the running sum of kept weights,
// `passed` before them, exceeds `past`.
__device__ int token_in(const SampleArgs &a, RowShared &sh, const float *row, int j0, int j1, u64 passed, u64 past,
                        Border border, float top, const Settings &s) {
    const int tid = threadIdx.x;
    for (; j0 < j1; j0 += kRow) {
        const int j = j0 + tid;
        u64 n = 0, all;
        if (j < j1) {
            const float z = gld(row + j);
            const double w = weight_of(z, top, s.per);
            if (border.keeps(float_key(z), j) && w >= s.least) n = steps_of(w, a.shift);
        }
        const u64 before = passed + block_scan<kRow>(sh.wave, n, &all);
        if (before <= past && before + n > past) sh.at = j;
        passed += all;
        if (passed > past) break;
    }
    __syncthreads();
    return sh.at;
}

__device__ __forceinline__ void done(const SampleArgs &a, int r, Border border, float top, double scale, int token) {
    if (threadIdx.x) return;
    RowState st{};
    st.kind = kDone;
    st.top = top;
    st.key = border.key;
    st.cut = border.cut;
    st.scale = scale;
    a.state[r] = st;
    if (a.tokens) gst(a.tokens + r, token);
}
__device__ __forceinline__ void failed(const SampleArgs &a, int r) {
    if (threadIdx.x) return;
    a.state[r].kind = kFailed;
    if (a.tokens) gst(a.tokens + r, -1);
}
__device__ __forceinline__ double number_of(const SampleArgs &a, int r) {
    const double u = a.tokens ? gld(a.u + r) : -1.0;
    return u >= 0.0 && u < 1.0 ? u : -1.0;
}

// A whole row by one workgroup: any case.
__device__ void slow_row(const SampleArgs &a, RowShared &sh, int r, float top, const Settings &s) {
    const float *row = row_of(a, r);
    const int tid = threadIdx.x;
    u64 n = 0, finite;
    for (int j = tid; j < a.V; j += kRow) n += gld(row + j) > -INFINITY;
    block_scan<kRow>(sh.wave, n, &finite);
    Border border = no_border();
    if (static_cast<u64>(s.k) < finite) select<false>(a, sh, row, top, s.per, static_cast<u64>(s.k), &border);
    auto sum_kept = [&](double least) {
        u64 sum = 0, all;
        for (int j = tid; j < a.V; j += kRow) {
            const float z = gld(row + j);
            if (!border.keeps(float_key(z), j)) continue;
            const double w = weight_of(z, top, s.per);
            if (w >= least) sum += steps_of(w, a.shift);
        }
        block_scan<kRow>(sh.wave, sum, &all);
        return all;
    };
    if (s.p < 1.0) {
        const u64 all = sum_kept(0.0);
        const double goal = ceil(s.p * static_cast<double>(all));
        select<true>(a, sh, row, top, s.per, goal < 1.0 ? 1 : min(static_cast<u64>(goal), all), &border);
    }
    const u64 total = sum_kept(s.least);
    const double u = number_of(a, r);
    const int token = u >= 0.0 ? token_in(a, sh, row, 0, a.V, 0, threshold(u, total), border, top, s) : -1;
    done(a, r, border, top, ldexp(1.0, a.shift) / static_cast<double>(total), token);
}

// ------------------------------------------------------------------ scan
// Values of a chunk as a thread holds them: quad i is the chunk's (i kScan +
// thread)-th.  Past the row's end: -inf.
struct Held {
    float z[kQuads][4];
    __device__ Held(const SampleArgs &a, const float *row, int c) {
        const int64_t base = static_cast<int64_t>(c) * kChunk;
        if (base + kChunk <= a.V) {
#pragma unroll
            for (int i = 0; i < kQuads; i++) {
                const f4u v = *(const SV_GLOBAL f4u *)(row + base + (i * kScan + threadIdx.x) * 4);
#pragma unroll
                for (int e = 0; e < 4; e++) z[i][e] = v[e];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kQuads; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int64_t j = base + (i * kScan + threadIdx.x) * 4 + e;
                    z[i][e] = j < a.V ? gld(row + j) : -INFINITY;
                }
        }
    }
};
// Places of a thread's chosen elements in the chunk's list, which is in the
// order of the indices.  bits[i]: chosen of quad i.  Returns their number.
struct Places {
    int at[kQuads];
};
__device__ __forceinline__ int places_of(u64 (*room)[2], const uint32_t (&bits)[kQuads], Places *out) {
    static_assert(kQuads == 8, "two words of four counts");
    u64 v[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kQuads; i++) v[i >> 2] += static_cast<u64>(__popc(bits[i])) << (16 * (i & 3));
    const int wave = threadIdx.x >> 6;
    const u64 upto[2] = {wave_scan(v[0]), wave_scan(v[1])};
    __syncthreads();
    if ((threadIdx.x & 63) == 63) {
        room[wave][0] = upto[0];
        room[wave][1] = upto[1];
    }
    __syncthreads();
    u64 before[2] = {0, 0}, sum[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < kScan / 64; w++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
            if (w == wave) before[k] = sum[k];
            sum[k] += room[w][k];
        }
    int at = 0;
#pragma unroll
    for (int i = 0; i < kQuads; i++) {
        const int k = i >> 2, by = 16 * (i & 3);
        out->at[i] = at + static_cast<int>((before[k] + upto[k] - v[k]) >> by & 0xFFFF);
        at += static_cast<int>(sum[k] >> by & 0xFFFF);
    }
    return at;
}
__device__ __forceinline__ void list_out(const SampleArgs &a, int slot, int c, const Held &h, const uint32_t (&bits)[kQuads],
                                         const Places &pl) {
    uint2 *list = a.lists + (static_cast<int64_t>(slot) * a.chunks + c) * a.cap;
#pragma unroll
    for (int i = 0; i < kQuads; i++) {
        int at = pl.at[i];
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (bits[i] >> e & 1) {
                if (at < a.cap) list[at] = make_uint2(__float_as_uint(h.z[i][e]), c * kChunk + (i * kScan + threadIdx.x) * 4 + e);
                at++;
            }
    }
}

// Elements that the list should have: some more than a top-k asks for.
__device__ __forceinline__ int list_target(const Settings &s, int V) { return s.k < V ? max(256, min(3000, s.k + s.k / 2 + 200)) : 1024; }

__global__ __launch_bounds__(kScan) void sample_scan_kernel(SampleArgs a) {
    __shared__ float s_sample[kScan / 64][64];
    __shared__ float s_tau, s_ref;
    __shared__ u64 s_room[kScan / 64][2];
    __shared__ double s_sum[kScan / 64];
    __shared__ float s_top[kScan / 64];
    __shared__ int s_rest;
    const int c = blockIdx.x, slot = blockIdx.y, r = a.row0 + slot, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (c == 0 && slot == 0 && tid == 0) a.flat[0] = 0;
    const float *row = row_of(a, r);
    const Settings s = settings_of(a, r);
    const Held h(a, row, c);

    // ---- the threshold: of 64 places of the row 64 values each (or of 8, or
    // one), the largest of every 64 (8, 1) that lie 64 apart; of these 64 the
    // one that the wanted part of the row's values should pass.
    const float part = static_cast<float>(list_target(s, a.V)) / static_cast<float>(a.V);
    const int of = part < 0.03f ? 64 : part < 0.2f ? 8 : 1;
    float most = -INFINITY;
    for (int i = wave; i < of; i += kScan / 64)
        most = fmaxf(most, gld(row + static_cast<int64_t>(i) * (a.V - 64) / of + lane));
    s_sample[wave][lane] = most;
    if (tid == 0) s_rest = 0;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < kScan / 64; w++) most = fmaxf(most, s_sample[w][lane]);
        const float none = powf(1.0f - part, static_cast<float>(of));
        const int nth = min(max(static_cast<int>(64.0f * (1.0f - none) + 0.5f), 1), 64) - 1;
        int rank = 0;
#pragma unroll
        for (int i = 0; i < 64; i++) {
            const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(most), i));
            rank += o > most || (o == most && i < lane);
        }
        if (rank == nth) s_tau = most;
        if (rank == 0) s_ref = most;
    }
    __syncthreads();
    const float tau = s_tau, ref = s_ref;

    // ---- the chunk
    float top = -INFINITY;
    bool bad = false, rest = false;
    uint32_t bits[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; i++) {
        bits[i] = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float z = h.z[i][e];
            top = fmaxf(top, z);
            bad |= !(z < INFINITY);
            const bool some = z > -INFINITY, listed = some && z >= tau;
            rest |= some && !listed;
            bits[i] |= static_cast<uint32_t>(listed) << e;
        }
    }
    double sum = -1.0;
    if (s.k == a.V && (s.p < 1.0 || s.least == 0.0)) {
        sum = 0.0;
#pragma unroll
        for (int i = 0; i < kQuads; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) sum += weight_of(h.z[i][e], ref, s.per);
        sum = wave_sum(sum);
    }
    top = wave_max(top);
    if (__any(bad)) top = NAN;
    rest = __any(rest);
    if (lane == 0) {
        s_sum[wave] = sum;
        s_top[wave] = top;
        if (rest) s_rest = 1;
    }
    Places pl;
    const int n = places_of(s_room, bits, &pl);  // its barriers: the waves' values are there
    list_out(a, slot, c, h, bits, pl);
    if (tid == 0) {
        ChunkRec rec{};
        rec.top = s_top[0];
        for (int w = 1; w < kScan / 64; w++) rec.top = rec.top != rec.top || s_top[w] != s_top[w] ? NAN : fmaxf(rec.top, s_top[w]);
        rec.n = n;
        rec.rest = s_rest;
        rec.tau = tau;
        rec.ref = ref;
        rec.sum = s_sum[0];
        for (int w = 1; w < kScan / 64; w++) rec.sum += sum < 0.0 ? 0.0 : s_sum[w];
        a.recs[static_cast<int64_t>(slot) * a.chunks + c] = rec;
    }
}

// ---------------------------------------------------------------- finish
// A list of a row, kPer entries a thread; entries past it are not `in`.
struct Listed {
    uint32_t key[kPer];
    int32_t j[kPer];
    bool in[kPer];
    float z[kPer];
};
// The chunks' lists one behind the other, through LDS: sh.offsets says where
// each begins.
__device__ __forceinline__ void take_lists(const SampleArgs &a, RowShared &sh, int slot, int n, Listed *out) {
    const int tid = threadIdx.x, lane = tid & 63;
    __syncthreads();
    for (int c = tid >> 6; c < a.chunks; c += kRow / 64) {
        const uint2 *list = a.lists + (static_cast<int64_t>(slot) * a.chunks + c) * a.cap;
        const int at = sh.offsets[c], of = sh.offsets[c + 1] - at;
        for (int i = lane; i < of; i += 64) {
            const uint2 v = gld8(list + i);
            sh.list.z[at + i] = __uint_as_float(v.x);
            sh.list.j[at + i] = static_cast<int32_t>(v.y);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int at = tid * kPer + i;
        out->in[i] = at < n;
        out->z[i] = at < n ? sh.list.z[at] : -INFINITY;
        out->j[i] = at < n ? sh.list.j[at] : 0;
        out->key[i] = float_key(out->z[i]);
    }
}
__device__ __forceinline__ u64 sum_of(RowShared &sh, const bool (&in)[kPer], const u64 (&amount)[kPer]) {
    u64 n = 0, all;
#pragma unroll
    for (int i = 0; i < kPer; i++) n += in[i] ? amount[i] : 0;
    block_scan<kRow>(sh.wave, n, &all);
    return all;
}

// The token of a row without filters: of the chunks' sums (`own`, `before`
// them and in all) the one that the number falls into, and in it the element.
__device__ int token_unfiltered(const SampleArgs &a, RowShared &sh, const float *row, double own, double before, double past,
                                float ref, double per) {
    constexpr int each = kChunk / kRow;
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) {
        sh.at = INT32_MAX;
        sh.last = 0;
    }
    __syncthreads();
    if (tid < a.chunks && before + own > past) atomicMin(&sh.at, tid);
    if (tid < a.chunks && own > 0.0) atomicMax(&sh.last, tid);
    __syncthreads();
    const int c = sh.at < INT32_MAX ? sh.at : sh.last;
    if (tid == c) sh.base = before;
    __syncthreads();
    if (tid == 0) {
        sh.at = INT32_MAX;
        sh.last = 0;
    }
    const double base = sh.base;
    const int64_t j0 = static_cast<int64_t>(c) * kChunk + tid * each;
    double w[each], mine = 0.0, all;
#pragma unroll
    for (int i = 0; i < each; i++) {
        w[i] = j0 + i < a.V ? weight_of(gld(row + j0 + i), ref, per) : 0.0;
        mine += w[i];
    }
    double upto = base + block_scan<kRow>(sh.wave_f, mine, &all);
#pragma unroll
    for (int i = each - 1; i >= 0; i--)
        if (w[i] > 0.0) {
            atomicMax(&sh.last, static_cast<int>(j0 + i));
            break;
        }
    bool found = false;
#pragma unroll
    for (int i = 0; i < each; i++) {
        upto += w[i];
        if (!found && w[i] > 0.0 && upto > past) {
            atomicMin(&sh.at, static_cast<int>(j0 + i));
            found = true;
        }
    }
    __syncthreads();
    return sh.at < INT32_MAX ? sh.at : sh.last;
}

// WHOLE: the row fits the registers and is its own list.
template <bool WHOLE>
__global__ __launch_bounds__(kRow) void sample_finish_kernel(SampleArgs a) {
    __shared__ RowShared sh;
    const int slot = blockIdx.x, r = a.row0 + slot, tid = threadIdx.x, lane = tid & 63;
    const float *row = row_of(a, r);
    const Settings s = settings_of(a, r);
    enum { kBad = 1, kOver = 2, kRest = 4 };

    // ---- what the chunks say, or the row itself
    Listed l;
    ChunkRec rec{};
    float top = -INFINITY;
    int flags = 0;
    u64 mine = 0;
    if (WHOLE) {
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            l.j[i] = tid * kPer + i;
            l.z[i] = l.j[i] < a.V ? gld(row + l.j[i]) : -INFINITY;
            l.in[i] = l.z[i] > -INFINITY;
            l.key[i] = float_key(l.z[i]);
            if (!(l.z[i] < INFINITY)) flags = kBad;
            top = fmaxf(top, l.z[i]);
            mine += l.in[i];
        }
    } else if (tid < a.chunks) {
        rec = a.recs[static_cast<int64_t>(slot) * a.chunks + tid];
        top = rec.top;
        flags = (rec.top != rec.top ? kBad : 0) | (rec.n > a.cap ? kOver : 0) | (rec.rest ? kRest : 0);
        mine = static_cast<u64>(rec.n);
    }
    if (tid == 0) {
        sh.flags = 0;
        sh.hi = 0;
    }
    __syncthreads();
    top = wave_max(top);
    if (lane == 0) atomicMax(&sh.hi, float_key(top));
    if (flags) atomicOr(&sh.flags, flags);
    u64 total;
    const u64 before = block_scan<kRow>(sh.wave, mine, &total);
    top = value_of(sh.hi);
    flags = sh.flags;
    if (!s.fine || (flags & kBad) || top == -INFINITY) {
        failed(a, r);
        return;
    }
    const bool usable = WHOLE || (!(flags & kOver) && total <= kList);
    const int n = usable ? static_cast<int>(total) : 0;
    const bool rest = !WHOLE && (!usable || (flags & kRest));
    double own = 0.0, sum_before = 0.0, sum = -1.0;
    float ref = 0.0f, tau = INFINITY;
    if (!WHOLE) {
        const ChunkRec &first = a.recs[static_cast<int64_t>(slot) * a.chunks];
        ref = gld(&first.ref);
        if (usable) tau = gld(&first.tau);
        own = tid < a.chunks ? rec.sum : 0.0;
        __syncthreads();
        sum_before = block_scan<kRow>(sh.wave_f, own, &sum);
        if (usable) {
            if (tid < a.chunks) sh.offsets[tid] = static_cast<int>(before);
            if (tid == 0) sh.offsets[a.chunks] = n;
            take_lists(a, sh, slot, n, &l);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; i++) {
                l.in[i] = false;
                l.z[i] = -INFINITY;
                l.key[i] = l.j[i] = 0;
            }
        }
    }
    const bool summed = sum > 0.0 && sum < INFINITY;
    double w[kPer];
    u64 steps[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        w[i] = weight_of(l.z[i], top, s.per);
        steps[i] = l.in[i] ? steps_of(w[i], a.shift) : 0;
    }

    // ---- the border, where it is in the list
    Border border = no_border();
    bool within = !rest;  // what is kept is in the list
    bool in[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) in[i] = l.in[i];
    auto cut_to = [&](Border b) {  // the narrower of the two: b tells apart only what is still in
        if (b.key > border.key) border = b;
        else if (b.key == border.key) border.cut = min(border.cut, b.cut);
#pragma unroll
        for (int i = 0; i < kPer; i++) in[i] = in[i] && border.keeps(l.key[i], l.j[i]);
    };
    // min-p alone keeps it in the list (weights are monotonic to a step or two of fp64)
    const bool low = weight_of(tau, top, s.per) * (1.0 + 1e-12) < s.least;
    int kind = kDone;
    u64 want = 0;
    if (s.k < n || (s.k == n && rest)) {
        if (s.k < n) cut_to(border_of<false>(sh, l.key, l.j, in, steps, static_cast<u64>(s.k)));
        within = true;
    } else if (rest && s.k < a.V) {
        if (s.p < 1.0) {
            kind = kSlow;
        } else if (!low) {
            kind = kByCount;
            want = static_cast<u64>(s.k);
        } else {
            within = true;
        }
    }
    if (kind == kDone && s.p < 1.0) {
        const u64 pool = sum_of(sh, in, steps);
        if (!within && !summed) {
            kind = kSlow;
        } else {
            const double goal = ceil(s.p * (within ? static_cast<double>(pool)
                                                   : sum * weight_of(ref, top, s.per) * ldexp(1.0, a.shift)));
            want = goal < 1.0 ? 1 : static_cast<u64>(goal);
            if (within) want = min(want, pool);
            if (want <= pool) {
                cut_to(border_of<true>(sh, l.key, l.j, in, steps, want));
                within = true;
            } else if (low) {
                within = true;
            } else {
                kind = kByMass;
            }
        }
    }
    const double u = number_of(a, r);
    if (kind == kDone && !within) {
        if (low) {
            within = true;
        } else if (s.least == 0.0 && summed) {
            const int token = u >= 0.0 ? token_unfiltered(a, sh, row, own, sum_before, u * sum, ref, s.per) : -1;
            done(a, r, no_border(), top, 1.0 / (sum * weight_of(ref, top, s.per)), token);
            return;
        } else {
            kind = kNoBorder;
        }
    }
    if (kind != kDone) {
        if (tid == 0) {
            RowState st{};
            st.kind = kind;
            st.top = top;
            st.want = want;
            a.state[r] = st;
            a.flat[1 + add_dev(a.flat, 1)] = slot;
        }
        a.bins[static_cast<int64_t>(slot) * kBins + tid] = 0;
        return;
    }

    // ---- the sum and the token
    u64 kept = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        if (!in[i] || !(w[i] >= s.least)) steps[i] = 0;
        kept += steps[i];
    }
    u64 all, upto = block_scan<kRow>(sh.wave, kept, &all);
    if (u >= 0.0) {
        const u64 past = threshold(u, all);
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            if (upto <= past && upto + steps[i] > past) sh.at = l.j[i];
            upto += steps[i];
        }
        __syncthreads();
    }
    done(a, r, border, top, ldexp(1.0, a.shift) / static_cast<double>(all), u >= 0.0 ? sh.at : -1);
}

// ------------------------------------------------------------- flat rows
__global__ __launch_bounds__(kScan) void sample_bins_kernel(SampleArgs a) {
    __shared__ u64 s_bins[kBins];
    const int items = gld(a.flat) * a.chunks;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int slot = gld(a.flat + 1 + it / a.chunks), c = it % a.chunks, r = a.row0 + slot;
        const int kind = gld(&a.state[r].kind);
        if (kind != kByCount && kind != kByMass) continue;
        const float top = gld(&a.state[r].top);
        const Settings s = settings_of(a, r);
        const Held h(a, row_of(a, r), c);
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kScan) s_bins[i] = 0;
        __syncthreads();
        const float scale = bin_scale(s.per);
#pragma unroll
        for (int i = 0; i < kQuads; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float z = h.z[i][e];
                if (!(z > -INFINITY)) continue;
                const u64 n = kind == kByCount ? 1 : steps_of(weight_of(z, top, s.per), a.shift);
                atomicAdd(&s_bins[bin_of(z, top, scale)], n);
            }
        __syncthreads();
        u64 *bins = a.bins + static_cast<int64_t>(slot) * kBins;
        for (int i = threadIdx.x; i < kBins; i += kScan)
            if (s_bins[i]) add_dev(bins + i, s_bins[i]);
    }
}

__global__ __launch_bounds__(kScan) void sample_gather_kernel(SampleArgs a) {
    __shared__ u64 s_room[kScan / 64][2], s_scan[kScan / 64], s_sum[kScan / 64], s_above;
    __shared__ int s_bin;
    const int items = gld(a.flat) * a.chunks, tid = threadIdx.x;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int slot = gld(a.flat + 1 + it / a.chunks), c = it % a.chunks, r = a.row0 + slot;
        const int kind = gld(&a.state[r].kind);
        if (kind == kSlow) continue;
        const float top = gld(&a.state[r].top);
        const u64 want = gld(&a.state[r].want);
        const Settings s = settings_of(a, r);
        const Held h(a, row_of(a, r), c);
        // the border's bin; past all of them if what is wanted is more than there is
        __syncthreads();
        if (tid == 0) {
            s_bin = kBins;
            s_above = 0;
        }
        __syncthreads();
        if (kind != kNoBorder) {
            const u64 *bins = a.bins + static_cast<int64_t>(slot) * kBins;
            const u64 b0 = gld(bins + 2 * tid), b1 = gld(bins + 2 * tid + 1);
            u64 all;
            const u64 before = block_scan<kScan>(s_scan, b0 + b1, &all);
            if (before < want && before + b0 >= want) {
                s_bin = 2 * tid;
                s_above = before;
            } else if (before + b0 < want && before + b0 + b1 >= want) {
                s_bin = 2 * tid + 1;
                s_above = before + b0;
            }
            __syncthreads();
        }
        const int bin = s_bin;
        const float scale = bin_scale(s.per);
        uint32_t bits[kQuads];
        u64 sum = 0;
#pragma unroll
        for (int i = 0; i < kQuads; i++) {
            bits[i] = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float z = h.z[i][e];
                if (!(z > -INFINITY)) continue;
                const int b = bin_of(z, top, scale);
                if (b == bin) bits[i] |= 1u << e;
                if (b >= bin) continue;
                const double w = weight_of(z, top, s.per);
                if (w >= s.least) sum += steps_of(w, a.shift);
            }
        }
        sum = wave_sum(sum);
        if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
        Places pl;
        const int n = places_of(s_room, bits, &pl);  // its barriers: the waves' sums are there
        list_out(a, slot, c, h, bits, pl);
        if (tid == 0) {
            ChunkRec rec{};
            rec.n = n;
            rec.steps = 0;
            for (int w = 0; w < kScan / 64; w++) rec.steps += s_sum[w];
            a.recs[static_cast<int64_t>(slot) * a.chunks + c] = rec;
            if (c == 0) {
                a.state[r].bin = bin;
                a.state[r].above = s_above;
            }
        }
    }
}

__global__ __launch_bounds__(kRow) void sample_settle_kernel(SampleArgs a) {
    __shared__ RowShared sh;
    const int tid = threadIdx.x;
    if (static_cast<int>(blockIdx.x) >= gld(a.flat)) return;
    const int slot = gld(a.flat + 1 + blockIdx.x), r = a.row0 + slot;
    const RowState st = a.state[r];
    const Settings s = settings_of(a, r);
    ChunkRec rec{};
    if (st.kind != kSlow && tid < a.chunks) rec = a.recs[static_cast<int64_t>(slot) * a.chunks + tid];
    u64 total;
    // a list that does not hold its chunk's elements counts as too many
    const u64 before = block_scan<kRow>(sh.wave, static_cast<u64>(rec.n > a.cap ? kList + 1 : rec.n), &total);
    if (st.kind == kSlow || total > kList) {
        slow_row(a, sh, r, st.top, s);
        return;
    }
    if (tid < a.chunks) sh.offsets[tid] = static_cast<int>(before);
    if (tid == 0) sh.offsets[a.chunks] = static_cast<int>(total);
    Listed l;
    take_lists(a, sh, slot, static_cast<int>(total), &l);
    u64 steps[kPer];
    double w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        w[i] = weight_of(l.z[i], st.top, s.per);
        steps[i] = l.in[i] ? steps_of(w[i], a.shift) : 0;
    }
    Border border = no_border();
    if (st.bin < kBins)
        border = st.kind == kByCount ? border_of<false>(sh, l.key, l.j, l.in, steps, st.want - st.above)
                                     : border_of<true>(sh, l.key, l.j, l.in, steps, st.want - st.above);
    // the chunks' kept sums
    __syncthreads();
    sh.hist[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; i++)
        if (l.in[i] && w[i] >= s.least && border.keeps(l.key[i], l.j[i])) atomicAdd(&sh.hist[l.j[i] / kChunk], steps[i]);
    __syncthreads();
    const u64 own = rec.steps + sh.hist[tid];
    u64 all;
    const u64 upto = block_scan<kRow>(sh.wave, own, &all);
    const double u = number_of(a, r);
    int token = -1;
    if (u >= 0.0) {
        const u64 past = threshold(u, all);
        if (upto <= past && upto + own > past) {
            sh.digit = tid;
            sh.above = upto;
        }
        __syncthreads();
        const int c = sh.digit;
        token = token_in(a, sh, row_of(a, r), c * kChunk, min(a.V, (c + 1) * kChunk), sh.above, past, border, st.top, s);
    }
    done(a, r, border, st.top, ldexp(1.0, a.shift) / static_cast<double>(all), token);
}

// --------------------------------------------------------------- outputs
__global__ __launch_bounds__(kScan) void sample_out_kernel(SampleArgs a) {
    const int c = blockIdx.x, r = a.row0 + blockIdx.y;
    const Settings s = settings_of(a, r);
    const Held h(a, row_of(a, r), c);
    const RowState st = a.state[r];
    const Border border{st.key, st.cut};
    const float none = st.kind == kFailed ? NAN : 0.0f, dropped = st.kind == kFailed ? NAN : -INFINITY;
    const int64_t base = static_cast<int64_t>(r) * a.V;
    const bool whole = (c + 1) * static_cast<int64_t>(kChunk) <= a.V;
#pragma unroll
    for (int i = 0; i < kQuads; i++) {
        const int64_t j = static_cast<int64_t>(c) * kChunk + (i * kScan + threadIdx.x) * 4;
        f4u p, k;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float z = h.z[i][e];
            bool keep = st.kind == kDone && z > -INFINITY && border.keeps(float_key(z), static_cast<int>(j) + e);
            double w = 0.0;
            if (keep) {
                w = weight_of(z, st.top, s.per);
                keep = w >= s.least;
            }
            p[e] = keep ? static_cast<float>(w * st.scale) : none;
            k[e] = keep ? z : dropped;
        }
        if (whole) {
            if (a.probs) *(SV_GLOBAL f4u *)(a.probs + base + j) = p;
            if (a.kept) *(SV_GLOBAL f4u *)(a.kept + base + j) = k;
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (j + e < a.V) {
                    if (a.probs) gst(a.probs + base + j + e, p[e]);
                    if (a.kept) gst(a.kept + base + j + e, k[e]);
                }
        }
    }
}

// ------------------------------------------------------------------ host
static int check_rows(int64_t rows, int64_t V) {
    SV_REQUIRE(rows >= 1 && rows <= kMaxRows, SV_ERR_SHAPE, "sample: rows must be in [1, 65535]");
    SV_REQUIRE(V >= 1 && V <= kMaxVocab, SV_ERR_SHAPE, "sample: V must be in [1, 2^24]");
    return SV_OK;
}

struct SamplePlan {
    int chunks, cap, slots;
    bool whole;
    size_t recs, lists, bins, flat, bytes;
};
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }
static SamplePlan sample_plan(int64_t rows, int64_t V) {
    SamplePlan p{};
    p.chunks = static_cast<int>((V + kChunk - 1) / kChunk);
    p.cap = std::max(1024, kList / p.chunks);
    p.whole = V <= kList;
    p.slots = static_cast<int>(std::min<int64_t>(rows, p.whole ? kMaxRows : kSlots));
    p.bytes = up256(static_cast<size_t>(rows) * sizeof(RowState));
    if (p.whole) return p;
    const size_t slots = static_cast<size_t>(p.slots), chunks = static_cast<size_t>(p.chunks);
    p.recs = p.bytes;
    p.lists = p.recs + up256(slots * chunks * sizeof(ChunkRec));
    p.bins = p.lists + up256(slots * chunks * static_cast<size_t>(p.cap) * sizeof(uint2));
    p.flat = p.bins + slots * kBins * sizeof(u64);
    p.bytes = p.flat + up256((slots + 1) * sizeof(int32_t));
    return p;
}

}  // namespace sv

using namespace sv;

extern "C" size_t sv_sample_workspace_bytes(int64_t rows, int64_t V) {
    if (check_rows(rows, V)) return 0;
    return sample_plan(rows, V).bytes;
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
    const SamplePlan p = sample_plan(rows, V);
    SV_REQUIRE(ws_bytes >= p.bytes, SV_ERR_WORKSPACE, "sample: workspace needs " + std::to_string(p.bytes) + " bytes");
    const size_t in = (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) + static_cast<size_t>(V)) * 4;
    const size_t out = static_cast<size_t>(rows) * static_cast<size_t>(V) * 4;
    SV_REQUIRE(!overlap(logits, in, probs, out) && !overlap(logits, in, kept, out) && !overlap(probs, out, kept, out), SV_ERR_ARG,
               "sample: probs, kept and logits overlap");
    int bits = 0;
    while ((1ll << bits) < V) bits++;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    SampleArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.params = params;
    a.per_row = n_params > 1;
    a.V = static_cast<int32_t>(V);
    a.shift = std::min(51, 63 - bits);
    a.chunks = p.chunks;
    a.cap = p.cap;
    a.u = u;
    a.tokens = tokens;
    a.probs = probs;
    a.kept = kept;
    a.state = reinterpret_cast<RowState *>(ws);
    a.recs = reinterpret_cast<ChunkRec *>(ws + p.recs);
    a.lists = reinterpret_cast<uint2 *>(ws + p.lists);
    a.bins = reinterpret_cast<u64 *>(ws + p.bins);
    a.flat = reinterpret_cast<int32_t *>(ws + p.flat);
    hipStream_t st = as_stream(stream);
    for (int64_t row0 = 0; row0 < rows; row0 += p.slots) {
        a.row0 = static_cast<int32_t>(row0);
        a.rows = static_cast<int32_t>(std::min<int64_t>(p.slots, rows - row0));
        const dim3 each(a.rows), pieces(p.chunks, a.rows);
        if (p.whole) {
            hipLaunchKernelGGL(sample_finish_kernel<true>, each, dim3(kRow), 0, st, a);
        } else {
            hipLaunchKernelGGL(sample_scan_kernel, pieces, dim3(kScan), 0, st, a);
            hipLaunchKernelGGL(sample_finish_kernel<false>, each, dim3(kRow), 0, st, a);
            const dim3 flat(std::min(kFlatGrid, a.rows * p.chunks));
            hipLaunchKernelGGL(sample_bins_kernel, flat, dim3(kScan), 0, st, a);
            hipLaunchKernelGGL(sample_gather_kernel, flat, dim3(kScan), 0, st, a);
            hipLaunchKernelGGL(sample_settle_kernel, each, dim3(kRow), 0, st, a);
        }
        if (probs || kept) hipLaunchKernelGGL(sample_out_kernel, pieces, dim3(kScan), 0, st, a);
    }
    return hip_check(hipGetLastError(), "sample launch");
}
