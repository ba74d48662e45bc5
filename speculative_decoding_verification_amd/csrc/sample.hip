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
// weight below half a step is never drawn: all of them together are at most V
// 2^-(s + 1) of the largest (2.2e-9 for 151936, 1.5e-5 for 2^24).  Sums over a
// whole row whose list does not hold it are fp64, of the weights as they are, in
// the order of its chunks: that of a row that nothing filters, and without a
// top-k the one that top-p is a share of.  That share is compared with sums of
// steps, so its border is off by what they leave out at most.
//
// One pass over the logits decides nearly every row:
//   scan    a workgroup per chunk of a row: a sample of the row gives a
//           threshold that about a thousand of its values pass; these are
//           listed in the order of their indices, with the chunk's largest
//           value and, if no top-k bounds what is kept, its sum of weights
//           (relative to the sample's largest value: the row's is not known);
//   finish  a workgroup per row: where what is kept lies within the list, the
//           border, the sum and the token come from the list in LDS; a row
//           without filters takes its token from the chunks' sums and one
//           chunk.
// A row whose kept set goes past the list (a flat distribution) is read twice
// more, by workgroups of one or two launches that find nothing to do otherwise:
//   bins    amounts (elements, or steps of weight) by the distance from the
//           largest value, which gives the border's bin;
//   gather  that bin's elements are listed and the kept weights above it
//           summed per chunk; the row's last workgroup settles it.
// What is left (a top-k past the list with a top-p as well, a bin of more
// elements than a list holds) is selected on the bits of z by that workgroup,
// in up to nine passes.
#include <algorithm>

#include "sv_internal.h"

namespace sv {

typedef unsigned long long u64;
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));  // rows may begin anywhere

constexpr int kThreads = 512;             // of a workgroup
constexpr int W = kThreads / 64;
constexpr int kQuads = 4;                // quads of a chunk that a thread holds
constexpr int kEach = kQuads * 4;        // elements
constexpr int kChunk = kThreads * kEach;
constexpr int kMaxChunks = (1 << 24) / kChunk;
constexpr int kList = 2560;              // listed elements that a row's workgroup holds
constexpr int kBins = 2048;
constexpr int kLevel = 512;              // parts that a range of keys is cut into
constexpr int kDigits = 2048;
constexpr int kSlots = 256;              // rows that are under way at once
constexpr int kFlatGrid = 512;           // workgroups of the passes over flat rows
constexpr int kOneLaunch = 256;
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
        u64 steps;   // gather: of the kept weights above the border's bin
    };
};

enum Kind { kWithin, kFailed, kByCount, kByMass, kNoBorder, kSlow };

// What the outputs of a row are made of, and what is known of a flat one.
struct RowState {
    int32_t kind;
    float top;
    uint32_t key;    // kept: keys above this one,
    int32_t cut;     // and those equal to it with a smaller index
    double scale;    // weight times this: probability
    u64 want;        // elements or steps to be kept
    float per_bin;   // bins to a unit of z, below top
    int32_t counted, gathered;  // chunks
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
    int32_t group;        // chunks of a scanning workgroup
    const double *u;
    int32_t *tokens;
    float *probs, *kept;
    RowState *state;  // [all rows]
    ChunkRec *recs;   // [slots][chunks]
    u64 *lists;       // [slots][chunks][cap]: bits of z, index in the high half
    u64 *bins;        // [slots][kBins]
    int32_t *flat;    // number of flat rows, of parts of their work taken, then their slots
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

// 2^y for y <= 1000 (relative error 2^-50; below 2^-1080: 0): y = n + f, |f| <=
// 1/2, 2^f = 1 + f q(f), and q of degree 9 through the ten Chebyshev points of
// that range, worked out in 60 digits.
__device__ __forceinline__ double exp2_of(double y) {
    constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52
    y = fmax(y, -1100.0);
    const double t = y + kRound, f = y - (t - kRound);
    double q = 7.070977866508139e-09;
    q = fma(q, f, 1.0205905413765595e-07);
    q = fma(q, f, 1.3215451633221434e-06);
    q = fma(q, f, 1.5252672924850737e-05);
    q = fma(q, f, 0.00015403530424776529);
    q = fma(q, f, 0.0013333558200794592);
    q = fma(q, f, 0.009618129107618665);
    q = fma(q, f, 0.05550410866465167);
    q = fma(q, f, 0.24022650695910075);
    q = fma(q, f, 0.6931471805599462);
    return ldexp(fma(q, f, 1.0), static_cast<int>(__double_as_longlong(t)));
}
__device__ __forceinline__ double weight_of(float z, float one, double per) {
    return exp2_of((static_cast<double>(z) - static_cast<double>(one)) * per);
}
// The same relative to the sample's largest value ref, in one rounding less:
// 2^(z per - hi) with hi = ref per as fp64 rounds it (shift_of = -hi), for (z -
// ref) per up to 1000.  What that rounding leaves, lo = ref per - hi, is in all
// weights of a row as a factor 2^lo, and with it in their sums: rest_of tells
// lo, exactly, to who compares such a sum with weights of the other form.
// per is taken by powers of two below what brings abs(ref) per to 2^51, so
// abs(lo) is at most an eighth: past that, values next to each other are 2^26
// apart in the exponent, and with less than their per the same weights stay 1
// and 0.
__device__ __forceinline__ double loose_per(float ref, double per) {
    return ldexp(per, min(51 - __builtin_amdgcn_frexp_exp(static_cast<double>(ref) * per), 0));
}
__device__ __forceinline__ double shift_of(float ref, double per) { return -(static_cast<double>(ref) * per); }
__device__ __forceinline__ double rest_of(float ref, double per) {
    return fma(static_cast<double>(ref), per, shift_of(ref, per));
}
__device__ __forceinline__ double loose_weight(float z, double per, double shift) {
    return exp2_of(fma(static_cast<double>(z), per, shift));
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
// Bin of a finite z; the last one holds all that is further.
__device__ __forceinline__ int bin_of(float z, float top, float per_bin) {
    return static_cast<int>(fminf((top - z) * per_bin, static_cast<float>(kBins - 1)));
}

__device__ __forceinline__ u64 entry_of(float z, int j) { return static_cast<u64>(j) << 32 | __float_as_uint(z); }

struct Border {
    uint32_t key;
    int32_t cut;
    __device__ bool keeps(uint32_t k, int j) const { return k > key || (k == key && j < cut); }
};
__device__ __forceinline__ Border no_border() { return Border{float_key(-INFINITY), 0}; }

// ------------------------------------------------- sums over a workgroup
// By moves within the registers (rows of 16 lanes, then across them): a lane
// exchange through LDS would wait for its six steps one by one.
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T moved(T v, T other) {  // `other` where the move gives no value
    constexpr int N = sizeof(T) / 4;
    uint32_t w[N], o[N];
    __builtin_memcpy(w, &v, sizeof(T));
    __builtin_memcpy(o, &other, sizeof(T));
#pragma unroll
    for (int i = 0; i < N; i++)
        w[i] = __builtin_amdgcn_update_dpp(static_cast<int>(o[i]), static_cast<int>(w[i]), CTRL, ROWS, 0xF, false);
    __builtin_memcpy(&v, w, sizeof(T));
    return v;
}
template <typename T>
__device__ __forceinline__ T lane_of(T v, int lane) {
    constexpr int N = sizeof(T) / 4;
    uint32_t w[N];
    __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
    for (int i = 0; i < N; i++) w[i] = __builtin_amdgcn_readlane(static_cast<int>(w[i]), lane);
    __builtin_memcpy(&v, w, sizeof(T));
    return v;
}
// v of the lanes up to and with this one, joined by f; none joins to nothing.
template <typename T, typename F>
__device__ __forceinline__ T wave_join(T v, T none, F f) {
    v = f(v, moved<0x111, 0xF>(v, none));  // row_shr 1, 2, 4, 8
    v = f(v, moved<0x112, 0xF>(v, none));
    v = f(v, moved<0x114, 0xF>(v, none));
    v = f(v, moved<0x118, 0xF>(v, none));
    v = f(v, moved<0x142, 0xA>(v, none));  // row_bcast 15, 31
    return f(v, moved<0x143, 0xC>(v, none));
}
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
    return wave_join(v, T(0), [](T a, T b) { return a + b; });
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
    return lane_of(wave_scan(v), 63);
}
__device__ __forceinline__ float wave_max(float v) {
    return lane_of(wave_join(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); }), 63);
}
// The same, NaN if one is NaN.
__device__ __forceinline__ float most_of(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float wave_most(float v) {
    return lane_of(wave_join(v, -INFINITY, [](float a, float b) { return most_of(a, b); }), 63);
}
__device__ __forceinline__ uint32_t wave_least(uint32_t v) {
    return lane_of(wave_join(v, ~0u, [](uint32_t a, uint32_t b) { return min(a, b); }), 63);
}
__device__ __forceinline__ int wave_or(int v) {
    return lane_of(wave_join(v, 0, [](int a, int b) { return a | b; }), 63);
}
// Sum over the threads before this one; *all is that over all.  `room` holds a
// value for each wave and is not in use.
template <typename T>
__device__ __forceinline__ T scan_once(T *room, T v, T *all) {
    const int wave = threadIdx.x >> 6;
    const T upto = wave_scan(v);
    if ((threadIdx.x & 63) == 63) room[wave] = upto;
    __syncthreads();
    T before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < W; w++) {
        if (w == wave) before = sum;
        sum += room[w];
    }
    *all = sum;
    return before + upto - v;
}
template <typename T>
__device__ __forceinline__ T block_scan(T *room, T v, T *all) {
    __syncthreads();
    return scan_once(room, v, all);
}

struct RowShared {
    union {
        struct {  // a list in the order of the indices
            uint32_t key[kList];
            uint32_t j[kList];  // kLow: the weight is below min_p
            u64 steps[kList + 1];
        };
        u64 hist[kDigits];  // amounts of bins or digits
    };
    // Amounts and numbers of the parts of a range, three in turn: a level
    // clears the next one's and has one barrier.
    u64 amount[3][kLevel];
    uint32_t number[3][kLevel];
    u64 wave[W], wave_n[W], wave_kept[W];
    double wave_f[W];
    float wave_top[W];
    uint32_t wave_low[W], wave_high[W];
    int32_t wave_flags[W], room[kQuads * W];
    u64 above;
    double base;
    int32_t digit, at, last;
    uint16_t offsets[kMaxChunks + 1];  // of the chunks' lists in this one
};
static_assert(sizeof(RowShared) <= 65536 && kBins <= kDigits, "LDS");
constexpr uint32_t kLow = 1u << 31;

// --------------------------------------- a border among listed elements
// Border of the first `want` (elements, or steps) of those of the n listed
// elements that `from` keeps, in falling order; want <= their sum, their keys
// in [lo, hi].  A level cuts the range into 512 parts; every wave finds the
// part with the border by itself.  *turn: which of the three parts' counts the
// next level uses, 0 at first, with amount[0] and number[0] cleared.
template <bool MASS>
__device__ Border border_of(RowShared &sh, int *turn, int n, Border from, u64 want, uint32_t lo, uint32_t hi) {
    constexpr int each = kLevel / 64;
    const int tid = threadIdx.x, lane = tid & 63;
    u64 above = 0;
    for (;;) {
        const int bits = hi > lo ? 32 - __clz(hi - lo) : 0, low = bits > 9 ? bits - 9 : 0;
        const int now = *turn, next = now == 2 ? 0 : now + 1;
        *turn = next;
        for (int i = tid; i < kLevel; i += kThreads) {
            sh.number[next][i] = 0;
            sh.amount[next][i] = 0;
        }
        for (int i = tid; i < n; i += kThreads) {
            const uint32_t k = sh.key[i];
            if (k >= lo && k <= hi && from.keeps(k, static_cast<int>(sh.j[i] & ~kLow))) {
                const int d = (k - lo) >> low;
                atomicAdd(&sh.number[now][d], 1u);
                if (MASS) atomicAdd(&sh.amount[now][d], sh.steps[i]);
            }
        }
        __syncthreads();
        // lane i: the parts from the (8 i)-th highest on
        u64 h[each], sum = 0;
#pragma unroll
        for (int i = 0; i < each; i++) {
            const int d = kLevel - 1 - lane * each - i;
            h[i] = MASS ? sh.amount[now][d] : sh.number[now][d];
            sum += h[i];
        }
        u64 before = above + wave_scan(sum) - sum;
        const int at = __ffsll(__ballot(before < want && before + sum >= want)) - 1;
        int d = 0;
        u64 of = 0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < each; i++) {
            if (!found && before + h[i] >= want) {
                found = true;
                d = kLevel - 1 - lane * each - i;
                of = h[i];
            }
            if (!found) before += h[i];
        }
        d = lane_of(d, at);
        above = lane_of(before, at);
        of = lane_of(of, at);
        const uint32_t number = sh.number[now][d];
        lo += static_cast<uint32_t>(d) << low;
        hi = min(hi, lo + ((1u << low) - 1));
        // one element, or all of the part's: nothing is left to be told apart
        if (low > 0 && (number == 1 || (!MASS && above + of == want))) return Border{lo, INT32_MAX};
        if (low > 0) continue;
        const u64 one = of / number, need = (want - above + one - 1) / one;
        if (need >= number) return Border{lo, INT32_MAX};
        // the first `need` of the equal ones
        const int per = (n + kThreads - 1) / kThreads, i0 = min(tid * per, n), i1 = min(i0 + per, n);
        u64 mine = 0, all;
        for (int i = i0; i < i1; i++) mine += sh.key[i] == lo && from.keeps(lo, static_cast<int>(sh.j[i] & ~kLow));
        u64 upto = block_scan(sh.wave, mine, &all);
        for (int i = i0; i < i1; i++) {
            const int j = static_cast<int>(sh.j[i] & ~kLow);
            if (sh.key[i] == lo && from.keeps(lo, j) && ++upto == need) sh.at = j + 1;
        }
        __syncthreads();
        const int cut = sh.at;
        __syncthreads();
        return Border{lo, cut};
    }
}

// The narrower of two borders, of which b tells apart only what a keeps.
__device__ __forceinline__ Border both(Border a, Border b) {
    return b.key > a.key ? b : Border{a.key, b.key == a.key ? min(a.cut, b.cut) : a.cut};
}

// --------------------------------------------------------- a row's chunks
// Values of a chunk as a thread holds them: quad i is the chunk's (i kThreads +
// thread)-th.  Every quad is one load, those at the row's end from its last
// four values; settle() then moves these to their places and puts -inf past
// the end (apart from the load: where the two meet, the loads are waited for).
struct Held {
    float z[kQuads][4];
    __device__ __forceinline__ void load(const SampleArgs &a, const float *row, int c) {
#pragma unroll
        for (int i = 0; i < kQuads; i++) {
            const uint32_t j = min(c * kChunk + (i * kThreads + static_cast<int>(threadIdx.x)) * 4, a.V - 4);
            const f4u v = *(const SV_GLOBAL f4u *)(reinterpret_cast<const uint8_t *>(row) + j * 4);
#pragma unroll
            for (int e = 0; e < 4; e++) z[i][e] = v[e];
        }
    }
    __device__ __forceinline__ void settle(const SampleArgs &a, int c) {
        if ((c + 1) * kChunk <= a.V) return;
#pragma unroll
        for (int i = 0; i < kQuads; i++) {
            const int left = a.V - (c * kChunk + (i * kThreads + static_cast<int>(threadIdx.x)) * 4);  // of the row
            const int by = 4 - min(max(left, 0), 4);
            const float v[4] = {z[i][0], z[i][1], z[i][2], z[i][3]};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float x = -INFINITY;
#pragma unroll
                for (int k = e; k < 4; k++) x = k - e == by ? v[k] : x;
                z[i][e] = x;
            }
        }
    }
};
// Places of a chunk's chosen elements in a list in the order of the indices.
// masks[i][e]: the wave's lanes whose element e of quad i is chosen; room: 32
// numbers; at[i]: the place of the lane's first one of quad i.  Returns how
// many there are; its barrier comes after every wave's work before the call.
typedef u64 Masks[kQuads][4];
__device__ __forceinline__ int places_of(const Masks &masks, int *room, int (&at)[kQuads]) {
    static_assert(kQuads * W <= 64, "a lane for each number");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < kQuads; i++) {
        const int number = __popcll(masks[i][0]) + __popcll(masks[i][1]) + __popcll(masks[i][2]) + __popcll(masks[i][3]);
        if (lane == i) room[i * W + wave] = number;
    }
    __syncthreads();
    const int own = lane < kQuads * W ? room[lane] : 0, upto = wave_scan(own);
#pragma unroll
    for (int i = 0; i < kQuads; i++) {
        at[i] = lane_of(upto - own, i * W + wave);
#pragma unroll
        for (int e = 0; e < 4; e++)
            at[i] += __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(masks[i][e] >> 32),
                                               __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(masks[i][e]), 0));
    }
    return lane_of(upto, 63);
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
        for (int i = tid; i < kDigits; i += kThreads) sh.hist[i] = 0;
        __syncthreads();
        for (int c = 0; c < a.chunks; c++) {
            Held h;
            h.load(a, row, c);
            h.settle(a, c);
#pragma unroll
            for (int i = 0; i < kQuads; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float z = h.z[i][e];
                    const uint32_t k = float_key(z);
                    if ((k & known) != prefix || !from.keeps(k, c * kChunk + (i * kThreads + tid) * 4 + e)) continue;
                    const u64 n = MASS ? steps_of(weight_of(z, top, per), a.shift) : 1;
                    atomicAdd(&sh.hist[(k >> low) & ((1u << bits) - 1)], n);
                }
        }
        __syncthreads();
        // digits in falling order
        constexpr int each = kDigits / kThreads;
        u64 h[each], sum = 0, all;
#pragma unroll
        for (int i = 0; i < each; i++) {
            h[i] = sh.hist[kDigits - 1 - each * tid - i];
            sum += h[i];
        }
        u64 before = above + block_scan(sh.wave, sum, &all);
#pragma unroll
        for (int i = 0; i < each; i++) {
            if (before < want && before + h[i] >= want) {
                sh.digit = kDigits - 1 - each * tid - i;
                sh.above = before;
            }
            before += h[i];
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
    static_assert(kEach <= 32, "a bit for each");
    for (int j0 = 0; j0 < a.V; j0 += kChunk) {  // a thread has consecutive ones
        const int own = j0 + tid * kEach;
        uint32_t is = 0;
#pragma unroll 4
        for (int i = 0; i < kEach; i++) {
            const uint32_t k = float_key(gld(row + min(own + i, a.V - 1)));
            is |= static_cast<uint32_t>(own + i < a.V && k == prefix && from.keeps(k, own + i)) << i;
        }
        u64 all;
        u64 run = passed + block_scan(sh.wave, static_cast<u64>(__popc(is)), &all);
        for (; is; is &= is - 1)
            if (++run == need) sh.at = own + __ffs(is);
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
// Steps of element j, if it is kept.
__device__ __forceinline__ u64 kept_steps(const SampleArgs &a, float z, int j, Border border, float top, const Settings &s) {
    const double w = weight_of(z, top, s.per);
    return border.keeps(float_key(z), j) && w >= s.least ? steps_of(w, a.shift) : 0;
}
// The first element of chunk c at which the running sum of kept weights,
// `passed` before the chunk, exceeds `past`; -1 if none does, *passed moved.
__device__ int token_in(const SampleArgs &a, RowShared &sh, const float *row, int c, u64 *passed, u64 past, Border border,
                        float top, const Settings &s) {
    const int first = c * kChunk, j0 = first + static_cast<int>(threadIdx.x) * kEach;
    u64 sum = 0, all;
#pragma unroll 4
    for (int i = 0; i < kEach; i++) {
        const float z = gld(row + min(j0 + i, a.V - 1));
        sum += j0 + i < a.V ? kept_steps(a, z, j0 + i, border, top, s) : 0;
    }
    const u64 run = *passed + block_scan(sh.wave, sum, &all);
    *passed += all;
    if (*passed <= past) return -1;
    if (run <= past && run + sum > past) {
        sh.at = threadIdx.x;
        sh.above = run;
    }
    __syncthreads();
    // that thread's elements, one a lane
    static_assert(kEach <= 64, "a lane for each element");
    const int at = first + sh.at * kEach, lane = threadIdx.x & 63, j = at + lane;
    const u64 own = lane < kEach && j < a.V ? kept_steps(a, gld(row + j), j, border, top, s) : 0;
    return at + __ffsll(__ballot(sh.above + wave_scan(own) > past)) - 1;
}

__device__ __forceinline__ void done(const SampleArgs &a, int r, Border border, float top, double scale, int token) {
    if (threadIdx.x) return;
    a.state[r] = RowState{kWithin, top, border.key, border.cut, scale, 0, 0.0f, 0, 0};
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
#pragma unroll 8
    for (int j = tid; j < a.V; j += kThreads) n += gld(row + j) > -INFINITY;
    block_scan(sh.wave, n, &finite);
    Border border = no_border();
    if (static_cast<u64>(s.k) < finite) select<false>(a, sh, row, top, s.per, static_cast<u64>(s.k), &border);
    auto sum_kept = [&](double least) {
        u64 sum = 0, all;
        for (int c = 0; c < a.chunks; c++) {
            Held h;
            h.load(a, row, c);
            h.settle(a, c);
#pragma unroll
            for (int i = 0; i < kQuads; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float z = h.z[i][e];
                    if (!border.keeps(float_key(z), c * kChunk + (i * kThreads + tid) * 4 + e)) continue;
                    const double w = weight_of(z, top, s.per);
                    if (w >= least) sum += steps_of(w, a.shift);
                }
        }
        block_scan(sh.wave, sum, &all);
        return all;
    };
    if (s.p < 1.0) {
        const u64 all = sum_kept(0.0);
        const double goal = ceil(s.p * static_cast<double>(all));
        select<true>(a, sh, row, top, s.per, goal < 1.0 ? 1 : min(static_cast<u64>(goal), all), &border);
    }
    const u64 total = sum_kept(s.least);
    const double u = number_of(a, r);
    int token = -1;
    u64 passed = 0;
    if (u >= 0.0)
        for (int c = 0; token < 0 && c < a.chunks; c++) token = token_in(a, sh, row, c, &passed, threshold(u, total), border, top, s);
    done(a, r, border, top, ldexp(1.0, a.shift) / static_cast<double>(total), token);
}

// ------------------------------------------------------------------ scan
// Elements that the list should have: a thousand, or 2.5 times what a top-k
// asks for (the threshold lets pass within 20 % or so of what it should).
__device__ __forceinline__ int list_target(const Settings &s, int V) { return s.k < V ? min(1600, 2 * s.k + s.k / 2 + 200) : 1024; }

// A workgroup takes `group` chunks one after the other; four of them share a
// compute unit, and one's loads pass while the others compute.
__global__ __launch_bounds__(kThreads, 8) void sample_scan_kernel(SampleArgs a) {
    __shared__ float s_sample[W][64];
    __shared__ float s_tau, s_ref;
    __shared__ int s_room[2][kQuads * (W)];
    __shared__ double s_sum[2][W];
    __shared__ float s_top[2][W];
    __shared__ int s_rest[2][W];
    const int slot = blockIdx.y, r = a.row0 + slot, tid = threadIdx.x, lane = tid & 63;
    const int c0 = blockIdx.x * a.group, c1 = min(c0 + a.group, a.chunks);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float *row = row_of(a, r);

    // ---- the threshold: of 64 places of the row (8, 1 in a short one) 64
    // values each, the largest of those that lie at the same offset; of these
    // 64 the one that the wanted part of the row's values should pass.
    const int few = a.V >= 32768 ? 6 : a.V >= 12288 ? 3 : 0, of = 1 << few;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int at = wave + i * (W);  // past the last place: the first again
        v[i] = gld(row + (static_cast<int64_t>(at < of ? at : 0) * (a.V - 64) >> few) + lane);
    }
    Held h;
    h.load(a, row, c0);
    const Settings s = settings_of(a, r);
    if (blockIdx.x == 0 && slot == 0 && tid < 2) a.flat[tid] = 0;
    float most = v[0];
#pragma unroll
    for (int i = 1; i < 8; i++) most = fmaxf(most, v[i]);
    s_sample[wave][lane] = most;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < W; w++) most = fmaxf(most, s_sample[w][lane]);
        if (!(most > -INFINITY)) most = -INFINITY;  // NaN: the row fails
        const float part = fminf(static_cast<float>(list_target(s, a.V)) / static_cast<float>(a.V), 0.999f);
        const float none = __builtin_amdgcn_exp2f(__builtin_amdgcn_logf(1.0f - part) * static_cast<float>(of));
        const int nth = min(max(static_cast<int>(64.0f * (1.0f - none) + 0.5f), 1), 64) - 1;
        int rank = 0;
#pragma unroll
        for (int i = 0; i < 64; i++) {
            const float o = lane_of(most, i);
            rank += o > most || (o == most && i < lane);
        }
        if (rank == nth) s_tau = most;
        if (rank == 0) s_ref = most;
    }
    __syncthreads();
    const float tau = s_tau, ref = s_ref, from = fmaxf(tau, -3.402823466e38f);  // finite ones alone
    const bool summed = s.k == a.V && (s.p < 1.0 || s.least == 0.0);
    const double per = loose_per(ref, s.per), less = shift_of(ref, per);

    // ---- the chunks
    for (int c = c0; c < c1; c++) {
        const int now = c & 1;
        if (c > c0) h.load(a, row, c);
        h.settle(a, c);
        float top = h.z[0][0];
#pragma unroll
        for (int i = 0; i < kQuads; i++) {
            top = most_of(most_of(top, h.z[i][0]), h.z[i][1]);
            top = most_of(most_of(top, h.z[i][2]), h.z[i][3]);
        }
        top = wave_most(top);
        if (!(top < INFINITY)) top = NAN;
        Masks masks;
#pragma unroll
        for (int i = 0; i < kQuads; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) masks[i][e] = __ballot(h.z[i][e] >= from);
        // any that are finite and not listed: most often the first ones tell
        bool rest = false;
#pragma unroll
        for (int e = 0; e < 4; e++) rest |= h.z[0][e] < from && h.z[0][e] > -INFINITY;
        int some = __any(rest);
        if (!some) {
#pragma unroll
            for (int i = 1; i < kQuads; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) rest |= h.z[i][e] < from && h.z[i][e] > -INFINITY;
            some = __any(rest);
        }
        double sum = -1.0;
        if (summed) {
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < kQuads; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) sum += loose_weight(h.z[i][e], per, less);
            sum = wave_sum(sum);
        }
        if (lane == 0) {
            s_sum[now][wave] = sum;
            s_top[now][wave] = top;
            s_rest[now][wave] = some;
        }
        int at[kQuads];
        const int n = places_of(masks, s_room[now], at);
        u64 *list = a.lists + (static_cast<int64_t>(slot) * a.chunks + c) * a.cap;
#pragma unroll
        for (int i = 0; i < kQuads; i++) {
            if (!(masks[i][0] | masks[i][1] | masks[i][2] | masks[i][3])) continue;
            const int j = c * kChunk + (i * kThreads + fresh(tid)) * 4;
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (h.z[i][e] >= from) {
                    if (at[i] < a.cap) list[at[i]] = entry_of(h.z[i][e], j + e);
                    at[i]++;
                }
        }
        if (tid == 0) {
            ChunkRec rec{};
            rec.top = s_top[now][0];
            rec.sum = s_sum[now][0];
            rec.rest = s_rest[now][0];
            for (int w = 1; w < W; w++) {
                rec.top = most_of(rec.top, s_top[now][w]);
                rec.sum += s_sum[now][w];
                rec.rest |= s_rest[now][w];
            }
            rec.n = n;
            rec.tau = tau;
            rec.ref = ref;
            a.recs[static_cast<int64_t>(slot) * a.chunks + c] = rec;
        }
    }
}

// ---------------------------------------------------------------- finish
// An element into a row's list.
__device__ __forceinline__ void enlist(const SampleArgs &a, RowShared &sh, int at, float z, int j, float top, const Settings &s) {
    const double w = weight_of(z, top, s.per);
    sh.key[at] = float_key(z);
    sh.steps[at] = steps_of(w, a.shift);
    sh.j[at] = static_cast<uint32_t>(j) | (w >= s.least ? 0u : kLow);
}
// The chunks' lists one behind the other (sh.offsets says where each begins, a
// barrier behind); a barrier ahead of their use.  Each chunk has as many
// threads, four of whose loads are on their way together.
__device__ __forceinline__ void take_lists(const SampleArgs &a, RowShared &sh, int slot, float top, const Settings &s) {
    int by = 6;
    while (by > 0 && a.chunks << by > kThreads) by--;
    const int of = 1 << by, first = threadIdx.x >> by, lane = threadIdx.x & (of - 1);
    for (int c = first; c < a.chunks; c += kThreads >> by) {
        const int begin = sh.offsets[c], n = sh.offsets[c + 1] - begin;
        const u64 *list = a.lists + (static_cast<int64_t>(slot) * a.chunks + c) * a.cap;
        for (int i0 = lane; i0 < n; i0 += 4 * of) {
            u64 v[4];
#pragma unroll
            for (int k = 0; k < 4; k++) v[k] = ld_dev(list + min(i0 + k * of, n - 1));
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (i0 + k * of < n)
                    enlist(a, sh, begin + i0 + k * of, __uint_as_float(static_cast<uint32_t>(v[k])), static_cast<int>(v[k] >> 32),
                           top, s);
        }
    }
}
// What of a list a border and min-p keep: steps of an element.
__device__ __forceinline__ u64 kept_of(const RowShared &sh, int i, Border border) {
    const uint32_t j = sh.j[i];
    return j < kLow && border.keeps(sh.key[i], static_cast<int>(j)) ? sh.steps[i] : 0;
}

// The token of a row without filters: of the chunks' sums the one that the
// number falls into, and in it the element.  A thread's chunks are [c0, c1),
// their sum `own` and that of those before them `before`.
__device__ int token_unfiltered(const SampleArgs &a, RowShared &sh, int slot, const float *row, int c0, int c1,
                                double own, double before, double past, float ref, double per) {
    constexpr int each = kEach;
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) {
        sh.at = INT32_MAX;
        sh.last = 0;
    }
    __syncthreads();
    // of those with a weight the first that passes it, or the last: the sums
    // before a thread's chunks and those before its elements are rounded in
    // different orders, so that none may, or one without any weight
    if (own > 0.0 && before + own > past) atomicMin(&sh.at, tid);
    if (own > 0.0) atomicMax(&sh.last, tid);
    __syncthreads();
    if (tid == (sh.at < INT32_MAX ? sh.at : sh.last)) {  // walks its chunks, in the same way
        int c = c0;
        double base = before, next = before;
        for (int i = c0; i < c1; i++) {
            const double sum = a.recs[static_cast<int64_t>(slot) * a.chunks + i].sum;
            if (sum == 0.0) continue;
            c = i;
            base = next;
            next += sum;
            if (next > past) break;
        }
        sh.digit = c;
        sh.base = base;
    }
    __syncthreads();
    if (tid == 0) {
        sh.at = INT32_MAX;
        sh.last = 0;
    }
    const double base = sh.base, less = shift_of(ref, per);
    const int first = sh.digit * kChunk, j0 = first + tid * each;
    double mine = 0.0, all;
    if (first + kChunk <= a.V) {
#pragma unroll 4
        for (int i = 0; i < each; i += 4) {
            const f4u z = *(const SV_GLOBAL f4u *)(row + j0 + i);
#pragma unroll
            for (int e = 0; e < 4; e++) mine += loose_weight(z[e], per, less);
        }
    } else {
#pragma unroll 4
        for (int i = 0; i < each; i++) {
            const float z = gld(row + min(j0 + i, a.V - 1));
            mine += j0 + i < a.V ? loose_weight(z, per, less) : 0.0;
        }
    }
    const double upto = base + block_scan(sh.wave_f, mine, &all);
    // the first thread that passes it; if roundings leave none, the last one
    // with a weight
    if (mine > 0.0 && upto + mine > past) atomicMin(&sh.at, tid);
    if (mine > 0.0) atomicMax(&sh.last, tid);
    __syncthreads();
    const int who = sh.at < INT32_MAX ? sh.at : sh.last;
    if (tid == who) sh.base = upto;
    __syncthreads();
    // its elements, one a lane
    static_assert(each <= 64, "a lane for each element");
    const int j = first + who * each + (tid & 63);
    const double w = (tid & 63) < each && j < a.V ? loose_weight(gld(row + j), per, less) : 0.0;
    const double run = sh.base + wave_scan(w);
    const u64 over = __ballot(w > 0.0 && run > past), some = __ballot(w > 0.0);
    return first + who * each + (over ? __ffsll(over) - 1 : 63 - __clzll(some));
}

// A value that a hundredth of a row's weights worth counting lie below: of 64
// places of the row 64 values each, the least of those at the same offset, and
// of these 64 the middle one.  Below 2^-64 of the largest nothing counts.
__device__ float bottom_of(const SampleArgs &a, RowShared &sh, const float *row, float top, double per) {
    float *least = reinterpret_cast<float *>(sh.hist);  // [waves][64]: the list has been used
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double from = static_cast<double>(top) - 64.0 / per;
    float low = INFINITY;
    for (int i = wave; i < 64; i += kThreads / 64) {
        const float z = gld(row + (static_cast<int64_t>(i) * (a.V - 64) >> 6) + lane);
        if (static_cast<double>(z) > from) low = fminf(low, z);
    }
    __syncthreads();
    least[threadIdx.x] = low;
    __syncthreads();
    for (int w = 0; w < kThreads / 64; w++) low = fminf(low, least[64 * w + lane]);
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < 64; i++) {
        const float o = lane_of(low, i);
        rank += o < low || (o == low && i < lane);
    }
    return lane_of(low, __ffsll(__ballot(rank == 32)) - 1);
}

// WHOLE: the row is its own list.
template <bool WHOLE>
__global__ __launch_bounds__(kThreads) void sample_finish_kernel(SampleArgs a) {
    __shared__ RowShared sh;
    const int slot = blockIdx.x, r = a.row0 + slot, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float *row = row_of(a, r);
    enum { kBad = 1, kOver = 2, kRest = 4 };

    // ---- what the chunks say, or the row itself
    float top = -INFINITY, ref = 0.0f, tau = INFINITY;
    uint32_t low = ~0u;
    int flags = 0;
    u64 mine = 0;
    double own = 0.0;
    const int span = (a.chunks + kThreads - 1) / kThreads, c0 = min(tid * span, a.chunks), c1 = min(c0 + span, a.chunks);
    const ChunkRec *recs = a.recs + static_cast<int64_t>(slot) * a.chunks;
    if (WHOLE) {
        for (int i = tid; i < a.V; i += kThreads) {
            const float z = gld(row + i);
            const uint32_t k = float_key(z);
            if (!(z < INFINITY)) flags = kBad;
            if (z > -INFINITY) {
                low = min(low, k);
                mine++;
            }
            top = fmaxf(top, z);
            sh.key[i] = k;
        }
    } else {
        ref = gld(&recs->ref);
        tau = gld(&recs->tau);
        for (int c = c0; c < c1; c++) {
            const ChunkRec rec = recs[c];
            top = fmaxf(top, rec.top);
            flags |= (rec.top != rec.top ? kBad : 0) | (rec.n > a.cap ? kOver : 0) | (rec.rest ? kRest : 0);
            mine += static_cast<u64>(rec.n);
            own += rec.sum;
        }
    }
    const Settings s = settings_of(a, r);
    const double u = number_of(a, r);
    int turn = 0;
    for (int i = tid; i < kLevel; i += kThreads) {
        sh.number[0][i] = 0;
        sh.amount[0][i] = 0;
    }
    top = wave_max(top);
    flags = wave_or(flags);
    if (WHOLE) low = wave_least(low);
    if (lane == 0) {
        sh.wave_top[wave] = top;
        sh.wave_flags[wave] = flags;
        sh.wave_low[wave] = low;
    }
    double sum = -1.0, sum_before = 0.0;
    if (!WHOLE) {
        const double upto = wave_scan(own);
        if (lane == 63) sh.wave_f[wave] = upto;
        sum_before = upto - own;
    }
    u64 total;
    const u64 before = scan_once(sh.wave_n, mine, &total);
#pragma unroll
    for (int w = 0; w < W; w++) {
        top = fmaxf(top, sh.wave_top[w]);
        flags |= sh.wave_flags[w];
        low = min(low, sh.wave_low[w]);
        if (!WHOLE) {
            if (w == 0) sum = 0.0;
            if (w == wave) sum_before += sum;
            sum += sh.wave_f[w];
        }
    }
    if (!s.fine || (flags & kBad) || top == -INFINITY) {
        failed(a, r);
        return;
    }
    const bool usable = WHOLE || (!(flags & kOver) && total <= kList);
    const bool rest = !WHOLE && (!usable || (flags & kRest));
    const bool summed = !WHOLE && sum > 0.0 && (static_cast<double>(top) - static_cast<double>(ref)) * s.per < 900.0;
    // the sum of all weights relative to the row's largest value
    const double sum_per = loose_per(ref, s.per);
    const double whole =
        summed ? sum * exp2_of((static_cast<double>(ref) - static_cast<double>(top)) * s.per - rest_of(ref, sum_per)) : 0.0;
    const int finite = usable ? static_cast<int>(total) : 0;  // listed
    const int n = WHOLE ? a.V : finite;                       // entries; -inf among them are below any border
    if (WHOLE) {
        for (int i = tid; i < n; i += kThreads) {
            const double w = weight_of(value_of(sh.key[i]), top, s.per);
            sh.steps[i] = steps_of(w, a.shift);
            sh.j[i] = static_cast<uint32_t>(i) | (w >= s.least ? 0u : kLow);
        }
    } else {
        if (usable) {
            int at = static_cast<int>(before);
            for (int c = c0; c < c1; c++) {
                sh.offsets[c] = static_cast<uint16_t>(at);
                at += recs[c].n;
            }
            if (tid == 0) sh.offsets[a.chunks] = static_cast<uint16_t>(n);
        }
        __syncthreads();
        if (usable) take_lists(a, sh, slot, top, s);
        low = float_key(fmaxf(tau, -3.402823466e38f));
    }
    __syncthreads();
    const uint32_t high = float_key(top);

    // ---- the border, where it is in the list
    Border border = no_border();
    bool within = !rest;  // what is kept is in the list
    // min-p alone keeps it in the list (weights are monotonic to a step or two of fp64)
    const bool short_of = usable && rest && weight_of(tau, top, s.per) * (1.0 + 1e-12) < s.least;
    Kind kind = kWithin;
    u64 want = 0;
    if (s.k < finite || (s.k == finite && rest)) {
        if (s.k < finite) {
            border = border_of<false>(sh, &turn, n, border, static_cast<u64>(s.k), low, high);
            low = max(low, border.key);
        } else {
            border = Border{low, INT32_MAX};  // the list: what passes its threshold
        }
        within = true;
    } else if (rest && s.k < a.V) {
        if (s.p < 1.0) {
            kind = kSlow;
        } else if (!short_of) {
            kind = kByCount;
            want = static_cast<u64>(s.k);
        } else {
            within = true;
        }
    }
    const int per = (n + kThreads - 1) / kThreads, i0 = min(tid * per, n), i1 = min(i0 + per, n);
    if (kind == kWithin && s.p < 1.0) {
        u64 pool = 0;
        for (int i = i0; i < i1; i++) pool += border.keeps(sh.key[i], static_cast<int>(sh.j[i] & ~kLow)) ? sh.steps[i] : 0;
        scan_once(sh.wave, pool, &pool);
        if (!within && !summed) {
            kind = kSlow;
        } else {
            const double goal = ceil(s.p * (within ? static_cast<double>(pool) : ldexp(whole, a.shift)));
            want = goal < 1.0 ? 1 : static_cast<u64>(goal);
            if (within) want = min(want, pool);
            if (want <= pool) {
                border = both(border, border_of<true>(sh, &turn, n, border, want, low, high));
                within = true;
            } else if (short_of) {
                within = true;
            } else {
                kind = kByMass;
            }
        }
    }
    if (kind == kWithin && !within) {
        if (short_of) {
            within = true;
        } else if (s.least == 0.0 && summed) {
            const int token = u >= 0.0 ? token_unfiltered(a, sh, slot, row, c0, c1, own, sum_before, u * sum, ref, sum_per) : -1;
            done(a, r, no_border(), top, 1.0 / whole, token);
            return;
        } else {
            kind = kNoBorder;
        }
    }
    if (kind != kWithin) {
        const float bottom = kind == kByCount || kind == kByMass ? bottom_of(a, sh, row, top, s.per) : 0.0f;
        if (tid == 0) {
            const float per_bin = static_cast<float>(kBins - 1) / fmaxf(top - bottom, 1e-30f);
            a.state[r] = RowState{kind, top, 0, 0, 0.0, want, per_bin, 0, 0};
            a.flat[2 + add_dev(a.flat, 1)] = slot;
        }
        for (int i = tid; i < kBins; i += kThreads) a.bins[static_cast<int64_t>(slot) * kBins + i] = 0;
        return;
    }

    // ---- the sum and the token
    u64 all, upto = 0;
    for (int i = i0; i < i1; i++) upto += kept_of(sh, i, border);
    upto = scan_once(sh.wave_kept, upto, &all);
    int token = -1;
    if (u >= 0.0) {
        const u64 past = threshold(u, all);
        for (int i = i0; i < i1; i++) {
            const u64 mass = kept_of(sh, i, border);
            if (upto <= past && upto + mass > past) sh.at = static_cast<int>(sh.j[i]);
            upto += mass;
        }
        __syncthreads();
        token = sh.at;
    }
    done(a, r, border, top, ldexp(1.0, a.shift) / static_cast<double>(all), token);
}

// ------------------------------------------------------------- flat rows
// Part `at` of `parts` of the flat rows' chunks: a run of them, so that what it
// needs of a row or leaves for it is fetched or written once.
struct Share {
    int at, end, slot, chunk, to;  // chunks [chunk, to) of the row
    __device__ Share(int items, int part, int parts) {
        const int each = items / parts, more = items % parts;
        at = each * part + min(part, more);
        end = at + each + (part < more);
    }
    __device__ bool next(const SampleArgs &a) {
        if (at >= end) return false;
        const int row = at / a.chunks;
        slot = gld(a.flat + 2 + row);
        chunk = at - row * a.chunks;
        to = min(a.chunks, chunk + end - at);
        at += to - chunk;
        return true;
    }
};

// Amounts of a row's chunks by the distance from its largest value.
__device__ void count_bins(const SampleArgs &a, RowShared &sh, const Share &share, const RowState &st, const Settings &s) {
    const int tid = threadIdx.x;
    const float *row = row_of(a, a.row0 + share.slot);
    Held h;
    h.load(a, row, share.chunk);
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int c = share.chunk; c < share.to; c++) {
        if (c > share.chunk) h.load(a, row, c);
        h.settle(a, c);
#pragma unroll
        for (int i = 0; i < kQuads; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float z = h.z[i][e];
                const u64 n = st.kind == kByCount ? 1 : steps_of(weight_of(z, st.top, s.per), a.shift);
                if (z > -INFINITY) atomicAdd(&sh.hist[bin_of(z, st.top, st.per_bin)], n);
            }
    }
    __syncthreads();
    u64 *bins = a.bins + static_cast<int64_t>(share.slot) * kBins;
    for (int i = tid; i < kBins; i += kThreads)
        if (sh.hist[i]) add_dev(bins + i, sh.hist[i]);
}

// A flat row whose chunks have all been gathered: `above` amounts lie above
// the border's bin (kBins: all elements do).
__device__ void settle_row(const SampleArgs &a, RowShared &sh, int slot, const RowState &st, const Settings &s, int bin, u64 above) {
    const int r = a.row0 + slot, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float *row = row_of(a, r);
    if (st.kind == kSlow) {
        slow_row(a, sh, r, st.top, s);
        return;
    }
    constexpr int span = kMaxChunks / kThreads;
    const ChunkRec *recs = a.recs + static_cast<int64_t>(slot) * a.chunks;
    int of[span];
    u64 own[span];  // kept steps of the thread's chunks
    u64 mine = 0, total;
#pragma unroll
    for (int k = 0; k < span; k++) {
        const int c = tid * span + k;
        of[k] = c < a.chunks ? ld_dev(&recs[c].n) : 0;
        own[k] = c < a.chunks ? ld_dev(&recs[c].steps) : 0;
        // a list that does not hold its chunk's elements counts as too many
        mine += static_cast<u64>(of[k] > a.cap ? kList + 1 : of[k]);
    }
    for (int i = tid; i < kLevel; i += kThreads) {
        sh.number[0][i] = 0;
        sh.amount[0][i] = 0;
    }
    const u64 before = block_scan(sh.wave_n, mine, &total);
    if (total > kList) {
        slow_row(a, sh, r, st.top, s);
        return;
    }
    const int n = static_cast<int>(total);
    int at = static_cast<int>(before);
#pragma unroll
    for (int k = 0; k < span; k++) {
        if (tid * span + k < a.chunks) sh.offsets[tid * span + k] = static_cast<uint16_t>(at);
        at += of[k];
    }
    if (tid == 0) sh.offsets[a.chunks] = static_cast<uint16_t>(n);
    __syncthreads();
    take_lists(a, sh, slot, st.top, s);
    __syncthreads();
    Border border = no_border();
    if (bin < kBins) {
        uint32_t low = ~0u, high = 0;
        for (int i = tid; i < n; i += kThreads) {
            low = min(low, sh.key[i]);
            high = max(high, sh.key[i]);
        }
        low = wave_least(low);
        high = ~wave_least(~high);
        if (lane == 0) {
            sh.wave_low[wave] = low;
            sh.wave_high[wave] = high;
        }
        __syncthreads();
        for (int w = 0; w < W; w++) {
            low = min(low, sh.wave_low[w]);
            high = max(high, sh.wave_high[w]);
        }
        int turn = 0;
        border = st.kind == kByCount ? border_of<false>(sh, &turn, n, border, st.want - above, low, high)
                                     : border_of<true>(sh, &turn, n, border, st.want - above, low, high);
    }
    // the kept steps of the list before each of its elements, in the place of its own
    const int per = (n + kThreads - 1) / kThreads, i0 = min(tid * per, n), i1 = min(i0 + per, n);
    u64 kept = 0, all;
    for (int i = i0; i < i1; i++) kept += kept_of(sh, i, border);
    u64 run = block_scan(sh.wave, kept, &all);
    for (int i = i0; i < i1; i++) {
        const u64 mass = kept_of(sh, i, border);
        sh.steps[i] = run;
        run += mass;
    }
    if (tid == 0) sh.steps[n] = all;
    __syncthreads();
    // the chunk, and in it the token
    u64 sum = 0;
#pragma unroll
    for (int k = 0; k < span; k++) {
        const int c = tid * span + k;
        if (c < a.chunks) own[k] += sh.steps[sh.offsets[c + 1]] - sh.steps[sh.offsets[c]];
        sum += own[k];
    }
    u64 upto = block_scan(sh.wave, sum, &all);
    const double u = number_of(a, r);
    int token = -1;
    if (u >= 0.0) {
        const u64 past = threshold(u, all);
#pragma unroll
        for (int k = 0; k < span; k++) {
            if (upto <= past && upto + own[k] > past) {
                sh.digit = tid * span + k;
                sh.above = upto;
            }
            upto += own[k];
        }
        __syncthreads();
        u64 passed = sh.above;
        token = token_in(a, sh, row, sh.digit, &passed, past, border, st.top, s);
    }
    done(a, r, border, st.top, ldexp(1.0, a.shift) / static_cast<double>(all), token);
}

// The border's bin of a flat row, and what lies above it; past all bins if what
// is wanted is more than there is.
__device__ __forceinline__ int border_bin(const SampleArgs &a, RowShared &sh, int slot, const RowState &st, u64 *above) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) {
        sh.digit = kBins;
        sh.above = 0;
    }
    __syncthreads();
    if (st.kind == kByCount || st.kind == kByMass) {
        constexpr int each = kBins / kThreads;
        const u64 *bins = a.bins + static_cast<int64_t>(slot) * kBins + tid * each;
        u64 b[each], sum = 0, all;
#pragma unroll
        for (int i = 0; i < each; i++) {
            b[i] = ld_dev(bins + i);
            sum += b[i];
        }
        u64 before = block_scan(sh.wave, sum, &all);
#pragma unroll
        for (int i = 0; i < each; i++) {
            if (before < st.want && before + b[i] >= st.want) {
                sh.digit = tid * each + i;
                sh.above = before;
            }
            before += b[i];
        }
        __syncthreads();
    }
    *above = sh.above;
    return sh.digit;
}

// Lists the border's bin of a row's chunks and sums the kept weights above it.
__device__ void gather(const SampleArgs &a, RowShared &sh, const Share &share, const RowState &st, const Settings &s, int bin) {
    const int tid = threadIdx.x;
    const float *row = row_of(a, a.row0 + share.slot);
    for (int c = share.chunk; c < share.to; c++) {
        Held h;
        h.load(a, row, c);
        h.settle(a, c);
        Masks masks;
        u64 sum = 0;
#pragma unroll
        for (int i = 0; i < kQuads; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float z = h.z[i][e];
                const int b = z > -INFINITY ? bin_of(z, st.top, st.per_bin) : kBins + 1;
                masks[i][e] = __ballot(b == bin);
                const double w = weight_of(z, st.top, s.per);
                if (b < bin && w >= s.least) sum += steps_of(w, a.shift);
            }
        sum = wave_sum(sum);
        __syncthreads();  // the last chunk's sums and numbers have been read
        if ((tid & 63) == 0) sh.wave_kept[tid >> 6] = sum;
        int at[kQuads];
        const int n = places_of(masks, sh.room, at);
        u64 *list = a.lists + (static_cast<int64_t>(share.slot) * a.chunks + c) * a.cap;
#pragma unroll
        for (int i = 0; i < kQuads; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (masks[i][e] >> (tid & 63) & 1) {
                    if (at[i] < a.cap) st_dev(list + at[i], entry_of(h.z[i][e], c * kChunk + (i * kThreads + tid) * 4 + e));
                    at[i]++;
                }
        if (tid == 0) {
            u64 steps = 0;
            for (int w = 0; w < W; w++) steps += sh.wave_kept[w];
            ChunkRec *rec = a.recs + static_cast<int64_t>(share.slot) * a.chunks + c;
            st_dev(&rec->n, n);
            st_dev(&rec->steps, steps);
        }
    }
}

// The passes over the flat rows: a launch each, or one (kBoth), where the call
// has at most kOneLaunch chunks.  That spares a call without flat rows 2 us and
// costs one whose rows are all flat the numbers' traffic (us, one launch against
// two, no flat row and all: 1 row of 151936 14.8 against 16.8 and 43.8 against
// 42.8; 48 rows of 33024 18.8 against 20.9 and 51.9 against 47.5; 32 rows of
// 151936, 608 chunks, all flat 83 against 67).  In one launch workgroups take
// parts of the work by a running number, first all parts of the counting, then
// all of the gathering.  Who gathers waits for the row's counting; its parts
// have lower numbers, so running workgroups have them, and these do not wait:
// the wait ends, however few workgroups run at once.  What one workgroup leaves
// for another is written through before the count that says so, and read where
// all see the same.  Two workgroups share a compute unit, at the price of a few
// registers that wait in memory while a row is settled (us, 64 and 256 flat rows
// of 151936: 43 and 103 for the gathering; one a unit 55 and 124).  Chunks go to
// workgroups in runs (dealt one by one 72 and 291, one a unit).
enum Pass { kCount, kGather, kBoth };
template <Pass PASS>
__global__ __launch_bounds__(kThreads, 4) void sample_flat_kernel(SampleArgs a) {
    __shared__ RowShared sh;
    __shared__ int s_part, s_last;
    const int items = gld(a.flat) * a.chunks, tid = threadIdx.x, parts = min(static_cast<int>(gridDim.x), items);
    if (static_cast<int>(blockIdx.x) >= parts) return;
    for (bool first = true;; first = false) {
        int part = blockIdx.x;
        if (PASS == kBoth) {
            __syncthreads();
            if (tid == 0) s_part = add_dev(a.flat + 1, 1);
            __syncthreads();
            part = s_part;
            if (part >= 2 * parts) break;
        } else if (!first) {
            break;
        }
        const bool counting = PASS == kCount || (PASS == kBoth && part < parts);
        Share share(items, PASS == kBoth && !counting ? part - parts : part, parts);
        while (share.next(a)) {
            const int slot = share.slot, r = a.row0 + slot, own = share.to - share.chunk;
            const RowState st = a.state[r];
            const Settings s = settings_of(a, r);
            const bool counted = st.kind == kByCount || st.kind == kByMass;
            if (counting) {
                if (!counted) continue;
                count_bins(a, sh, share, st, s);
                if (PASS == kBoth) {
                    drain();
                    __syncthreads();
                    if (tid == 0) add_dev(&a.state[r].counted, own);
                }
                continue;
            }
            if (PASS == kBoth && counted) {
                if (tid == 0)
                    while (ld_dev(&a.state[r].counted) != a.chunks) __builtin_amdgcn_s_sleep(4);
                __syncthreads();
            }
            u64 above;
            const int bin = border_bin(a, sh, slot, st, &above);
            if (st.kind != kSlow) gather(a, sh, share, st, s, bin);
            drain();
            __syncthreads();
            if (tid == 0) s_last = add_dev(&a.state[r].gathered, own) == a.chunks - own;
            __syncthreads();
            if (s_last) settle_row(a, sh, slot, st, s, bin, above);
        }
    }
}

// --------------------------------------------------------------- outputs
// Stored past the L2: a launch's outputs pass what it holds (us, 256 rows of
// 151936 with probs and kept 120 -> 104, 48 of 33024 22.3 -> 21.2, 5 the same).
constexpr int kOut = 256, kOutPiece = kOut * 8;
__global__ __launch_bounds__(kOut) void sample_out_kernel(SampleArgs a) {
    const int r = a.row0 + blockIdx.y;
    const float *row = row_of(a, r);
    const int j0 = blockIdx.x * kOutPiece + threadIdx.x * 4;
    float z[2][4];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int j = j0 + i * kOut * 4;
        if (j + 4 <= a.V) {
            const f4u v = *(const SV_GLOBAL f4u *)(row + j);
#pragma unroll
            for (int e = 0; e < 4; e++) z[i][e] = v[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) z[i][e] = j + e < a.V ? gld(row + j + e) : -INFINITY;
        }
    }
    const RowState st = a.state[r];
    const Settings s = settings_of(a, r);
    const Border border{st.key, st.cut};
    const float none = st.kind == kFailed ? NAN : 0.0f, dropped = st.kind == kFailed ? NAN : -INFINITY;
    const int64_t base = static_cast<int64_t>(r) * a.V;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int j = j0 + i * kOut * 4;
        f4u p, k;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            bool keep = st.kind != kFailed && z[i][e] > -INFINITY && border.keeps(float_key(z[i][e]), j + e);
            double w = 0.0;
            if (keep) {
                w = weight_of(z[i][e], st.top, s.per);
                keep = w >= s.least;
            }
            p[e] = keep ? static_cast<float>(w * st.scale) : none;
            k[e] = keep ? z[i][e] : dropped;
        }
        if (j + 4 <= a.V) {
            if (a.probs) __builtin_nontemporal_store(p, (SV_GLOBAL f4u *)(a.probs + base + j));
            if (a.kept) __builtin_nontemporal_store(k, (SV_GLOBAL f4u *)(a.kept + base + j));
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
    p.bins = p.lists + up256(slots * chunks * static_cast<size_t>(p.cap) * sizeof(u64));
    p.flat = p.bins + slots * kBins * sizeof(u64);
    p.bytes = p.flat + up256((slots + 2) * sizeof(int32_t));
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
    a.lists = reinterpret_cast<u64 *>(ws + p.lists);
    a.bins = reinterpret_cast<u64 *>(ws + p.bins);
    a.flat = reinterpret_cast<int32_t *>(ws + p.flat);
    hipStream_t st = as_stream(stream);
    for (int64_t row0 = 0; row0 < rows; row0 += p.slots) {
        a.row0 = static_cast<int32_t>(row0);
        a.rows = static_cast<int32_t>(std::min<int64_t>(p.slots, rows - row0));
        const dim3 each(a.rows);
        if (p.whole) {
            hipLaunchKernelGGL(sample_finish_kernel<true>, each, dim3(kThreads), 0, st, a);
        } else {
            // four workgroups a compute unit, if the rows give that many
            a.group = std::max(1, (a.rows * p.chunks + 1023) / 1024);
            hipLaunchKernelGGL(sample_scan_kernel, dim3((p.chunks + a.group - 1) / a.group, a.rows), dim3(kThreads), 0, st, a);
            hipLaunchKernelGGL(sample_finish_kernel<false>, each, dim3(kThreads), 0, st, a);
            const dim3 flat(std::min(kFlatGrid, a.rows * p.chunks));
            if (a.rows * p.chunks <= kOneLaunch) {
                hipLaunchKernelGGL(sample_flat_kernel<kBoth>, flat, dim3(kThreads), 0, st, a);
            } else {
                hipLaunchKernelGGL(sample_flat_kernel<kCount>, flat, dim3(kThreads), 0, st, a);
                hipLaunchKernelGGL(sample_flat_kernel<kGather>, flat, dim3(kThreads), 0, st, a);
            }
        }
        if (probs || kept)
            hipLaunchKernelGGL(sample_out_kernel, dim3(static_cast<unsigned>((V + kOutPiece - 1) / kOutPiece), a.rows), dim3(kOut), 0,
                               st, a);
    }
    return hip_check(hipGetLastError(), "sample launch");
}
