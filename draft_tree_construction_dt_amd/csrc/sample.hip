// dt_sample_rows: a token for every row of logits, drawn by a given random
// number among those that top-k, top-p and min-p leave.
//
// What stays is a beginning of the order (logit desc, id asc): all tokens above
// some logit, and the first few by id of those at it.  With the weights held as
// integers (w scaled by 2^shift, so that V of them fit 62 bits) every sum is
// exact, whatever its order and grouping: the cut can be narrowed digit by digit
// over the logits' bits with histograms in LDS, the drawn token over the ids, and
// neither ever meets two sums that should agree and do not.
//
// A workgroup takes a row.  It reads it for the largest logit, and keeps each
// thread's own two largest: the j-th of those is a limit that j tokens at least
// reach.  Then, by what the request asks for:
//   top-k       the tokens at or above that limit go to a list in LDS, once
//               through the row, and all else happens there;
//   min-p only  the same with the limit that min_p sets;
//   top-p       one pass makes every weight and a histogram of them over the
//               logits, and the list: usually the cut lies within it.  If not
//               (a flat row), the tokens of the cut's own bin are listed, and
//               a last pass draws among all;
//   none        one pass for the sums of 16 parts of the row, then the part's
//               parts.
// A list that overflows, or a larger top_k, narrows the cut over the row itself.
//
// Measured: 512 rows of 151936 bf16 (156 MB; a copy's rate would take 32 us) in
// 28 us where all are greedy, 60-64 with top-k 20-50, 72 with temperature alone,
// 85 with min-p, 93 with top-k 1000, 129-131 with top-p; every kind of setting
// among them 126-129.  All of these rows are resident at once, two a compute
// unit, so a mixed batch lasts as long as its slowest row: a compute unit has work
// 55% of the time and vector units are busy 32% (77% and 52% where all rows have
// top-p, whose waves spend 55% of their time waiting for memory and LDS).  One row
// of 32000 fp32 20 us, the latency of its passes.  A workgroup of 1024 threads a row took
// 17 us for the one row and 164 for the 512.
#include <float.h>
#include <math.h>

#include "pass.h"
#include "wave.h"

namespace dt {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512, kWaves = kThreads / 64;      // two workgroups on a compute unit
constexpr int kBits = 11, kBins = 1 << kBits;              // of a histogram
// Tokens of the list: what the LDS of two workgroups leaves.  (512 rows of 151936
// with top_k 1000: 94 us with 4096 as with 6144; 2048 overflow, 340 us and more.)
constexpr int kList = 6144;
// How many of the threads' two largest logits reach the list's limit.  For top_k
// as many as that; a workgroup has 1024 of them, and the largest usual top_k is
// 1000.  Larger ones go by counted values or over the row (512 rows of 151936,
// top_k 1000: 88 us by list, 130 by counted bf16 values; fp32 122 by list, 354 over
// the row; one row of 32000: 26 and 28, fp32 29 and 53; smaller top_k gain more).
constexpr int kMostK = 1000;
// For top_p alone (fp32) a fixed number.  512 rows of 151936, top_p 0.9, with 224,
// 448, 896, 1000: 325, 329, 338, 342 us; one row of 32000: 35, 36, 39, 41.
constexpr int kForP = 896;
constexpr int kTable = 64;
// Tokens of a list whose pairs are compared.  512 rows of 151936 bf16 with 64, 128,
// 256, 512: top_k 50 60, 61, 64, 67 us, 100 71, 65, 70, 78, 200 72, 72, 84, 98,
// min_p 0.05 67, 67, 85, 152.
constexpr int kShort = 256;
constexpr unsigned kMaxGridX = 1 << 20;

// Bits whose order is that of the values (no NaN; -0 and 0 are one).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// e^((x - top) / temperature) * 2^shift, rounded: 2^(j / 64) from a table in LDS
// times the series of 2^f, |f| <= 1/128, to the fourth power; the next term is
// below 2^-44.  In fp64: a sum over V weights is compared with u times the total,
// and errors of 2^-24 a weight would move the drawn token in one row of a
// thousand.  No branches: eight logits' weights are made side by side.
typedef const __attribute__((address_space(3))) double* Table;
struct Weights {
    double top, rate;              // rate = 64 log2(e) / temperature
    double least;                  // 64 times the smallest exponent of a weight
    Table table;                   // 2^(j / 64 + shift)

    __device__ __forceinline__ u64 operator()(float x) const {
        constexpr double kRound = 6755399441055744.0, kOne = 0.69314718055994530942 / kTable;
        constexpr double k2 = kOne * kOne / 2, k3 = k2 * kOne / 3, k4 = k3 * kOne / 4;
        const double y = ((double)x - top) * rate, t = y > least ? y : least;      // (NaN, as inf - inf: the least)
        const double r = t + kRound, f = t - (r - kRound);
        const int i = (int)(uint32_t)__double_as_longlong(r);
        const u64 e = (u64)__double_as_longlong(table[i & (kTable - 1)]) + ((u64)(uint32_t)(i >> 6) << 52);
        const double w = __longlong_as_double((long long)e);
        const double q = f * (kOne + f * (k2 + f * (k3 + f * k4)));
        return (u64)__double_as_longlong(fma(w, q, w) + 4503599627370496.0) & 0xFFFFFFFFFFFFFull;
    }
};

// One row in memory, in groups of 16 aligned bytes; what the first and the last
// group hold beside the row comes as -inf.  NaN come as they are from load() and
// groups_of(), and as -inf from scan() and each(): they count as -inf everywhere.
template <class E>
struct Row {
    static constexpr int kEach = 16 / sizeof(E);
    static constexpr uint32_t kNone = sizeof(E) == 2 ? 0xFF80FF80u : 0xFF800000u;
    typedef const __attribute__((address_space(1))) E* Elements;
    typedef const __attribute__((address_space(1))) u32x4* Vectors;
    Elements base;                 // of group 0
    int before, V, groups;         // elements of group 0 that are not the row's

    __device__ __forceinline__ Row(const void* logits, int64_t row, int V_) : V(V_) {
        const int64_t at = row * V_;
        before = (int)(at % kEach);
        base = (Elements)((const E*)logits + (at - before));
        groups = (int)(((int64_t)before + V_ + kEach - 1) / kEach);
    }
    static __device__ __forceinline__ float get(uint32_t bits) {
        return sizeof(E) == 2 ? __uint_as_float(bits << 16) : __uint_as_float(bits);
    }
    __device__ __forceinline__ u32x4 load(int g) const {
        if (g > 0 && g < groups - 1) return *(Vectors)(base + (int64_t)g * kEach);
        u32x4 v = {kNone, kNone, kNone, kNone};
        for (int e = 0; e < kEach; ++e) {
            const int64_t id = (int64_t)g * kEach - before + e;
            if (id < 0 || id >= V) continue;
            const uint32_t b = base[(int64_t)g * kEach + e];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(E) == 2) {
                    if (e == 2 * i) v[i] = (v[i] & 0xFFFF0000u) | b;
                    if (e == 2 * i + 1) v[i] = (v[i] & 0xFFFFu) | b << 16;
                } else if (e == i) {
                    v[i] = b;
                }
            }
        }
        return v;
    }
    static __device__ __forceinline__ float at(const u32x4& v, int e) {
        if constexpr (sizeof(E) == 2) return __uint_as_float(e & 1 ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16);
        else return __uint_as_float(v[e]);
    }
    // f(g, v) for groups g0 .. g1 - 1 by one wave, whose lanes stay together
    // (f may use the whole wave; lanes without a group get -inf).
    // DEEP loads of a lane are in flight.
    template <int DEEP, class F>
    __device__ __forceinline__ void groups_of(int g0, int g1, int lane, F f) const {
        for (int64_t first = g0; first < g1; first += DEEP * 64) {
            u32x4 v[DEEP];
#pragma unroll
            for (int i = 0; i < DEEP; ++i) {
                const int64_t g = first + i * 64 + lane;
                v[i] = u32x4{kNone, kNone, kNone, kNone};
                if (g < g1) v[i] = load((int)g);
            }
#pragma unroll
            for (int i = 0; i < DEEP; ++i) {
                if (first + i * 64 >= g1) break;
                f((int)(first + i * 64) + lane, v[i]);
            }
        }
    }
    // f(id, x) for every element of them.
    template <class F>
    __device__ __forceinline__ void scan(int g0, int g1, int lane, F f) const {
        groups_of<4>(g0, g1, lane, [&](int g, const u32x4& v) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const float x = at(v, e);
                f(g * kEach - before + e, x == x ? x : -INFINITY);
            }
        });
    }
    // the whole row, a part each wave
    template <class F>
    __device__ __forceinline__ void each(int wave, int lane, F f) const {
        const int per = (groups + kWaves - 1) / kWaves, g0 = wave * per < groups ? wave * per : groups;
        scan(g0, g0 + per < groups ? g0 + per : groups, lane, f);
    }
};

// Weights of the 16-bit type's values, and how often they occur: 22 binades of
// magnitudes (of 128 values) that reach past every logit that weighs anything,
// positive ones, then negative ones.
constexpr int kBinades = 22, kMagnitudes = kBinades * 128;
struct Values {
    u64 weight[2 * kMagnitudes];
    uint32_t count[2 * kMagnitudes];
};
struct Histogram {
    u64 weight[kBins];
    uint32_t count[kBins];
    float list[kList];
    int ids[kList];
};
struct Shared {
    union {                        // a row goes by one or the other
        Histogram h;
        Values v;
    };
    double table[kTable];
    u64 wave[2][kWaves];
    u64 found[4];
    u64 tiny_weight;               // of magnitudes smaller than those of `v`
    uint32_t tiny_count;
    uint32_t listed;
};
static_assert(sizeof(Shared) <= 80 * 1024, "two workgroups on a compute unit");

// The list, once it is complete.
struct List {
    const Shared& s;
    int n;

    template <class F>
    __device__ __forceinline__ void each(int wave, int lane, F f) const {
        for (int i = wave * 64 + lane; i < n; i += kThreads) f(s.h.ids[i], s.h.list[i]);
    }
};

__device__ __forceinline__ u64 wave_add_u64(u64 v) {
#pragma unroll
    for (int s = 0; s < 4; ++s) v += dpp_step64(v, s);
    return (readlane64(v, 0) + readlane64(v, 16)) + (readlane64(v, 32) + readlane64(v, 48));
}
template <int CTRL>
__device__ __forceinline__ u64 shifted(u64 v) {            // within the rows of 16 lanes; 0 from outside
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xF, 0xF, false);
    return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 wave_prefix_u64(u64 v, int lane) {
    v += shifted<0x111>(v);                                // row_shr:1, 2, 4, 8
    v += shifted<0x112>(v);
    v += shifted<0x114>(v);
    v += shifted<0x118>(v);
    const u64 a = readlane64(v, 15), b = readlane64(v, 31), c = readlane64(v, 47);
    return v + (lane >= 16 ? a : 0) + (lane >= 32 ? b : 0) + (lane >= 48 ? c : 0);
}
__device__ __forceinline__ u64 block_add(u64 v, Shared& s, int wave, int lane) {
    v = wave_add_u64(v);
    if (lane == 0) s.wave[0][wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += s.wave[0][i];
    __syncthreads();
    return v;
}

// Where a beginning of some order ends: at this key, above which lie `count`
// tokens of `weight` in all; `ties` tokens are at it.
struct Cut {
    uint32_t key;
    uint32_t count, ties;
    u64 weight;
};

// The bin, from the top, with which the tokens' number (or weight) reaches
// `limit`, which all of them do; counts and weights before it go to `cut`.
template <bool BY_WEIGHT>
__device__ __forceinline__ int pick_bin(int bins, u64 limit, Cut& cut, Shared& s, int wave, int lane) {
    // thread t's bins are the t-th kMine from the top
    constexpr int kMine = kBins / kThreads;
    const int top = bins - 1 - kMine * (wave * 64 + lane);
    u64 c[kMine], w[kMine], cs = 0, ws = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        c[i] = top - i >= 0 ? s.h.count[top - i] : 0;
        w[i] = BY_WEIGHT && top - i >= 0 ? s.h.weight[top - i] : 0;
        cs += c[i];
        ws += w[i];
    }
    const u64 cp = wave_prefix_u64(cs, lane), wp = BY_WEIGHT ? wave_prefix_u64(ws, lane) : 0;
    if (lane == 63) {
        s.wave[0][wave] = cp;
        s.wave[1][wave] = wp;
    }
    __syncthreads();
    u64 cx = cut.count + cp - cs, wx = cut.weight + wp - ws;       // before this thread's bins
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i) {
        cx += i < wave ? s.wave[0][i] : 0;
        if (BY_WEIGHT) wx += i < wave ? s.wave[1][i] : 0;
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const u64 m = BY_WEIGHT ? wx : cx;
        if (m < limit && m + (BY_WEIGHT ? w[i] : c[i]) >= limit) {
            s.found[0] = (u64)(top - i);
            s.found[1] = cx;
            s.found[2] = wx;
            s.found[3] = c[i];
        }
        cx += c[i];
        wx += w[i];
    }
    __syncthreads();
    cut.count = (uint32_t)s.found[1];
    cut.weight = s.found[2];
    cut.ties = (uint32_t)s.found[3];
    return (int)s.found[0] & (kBins - 1);
}

__device__ __forceinline__ void clear_bins(int bins, Shared& s, int tid) {
    for (int i = tid; i < bins; i += kThreads) {
        s.h.count[i] = 0;
        s.h.weight[i] = 0;
    }
    __syncthreads();
}

// The first key, from the top, with which the number (or weight) of the tokens
// of `from` that weigh something reaches `limit`, which all of them do.
// of(id, x, key, weight) says which those are, and their keys, whose bits from
// `bits` on are those of `prefix`.
template <bool BY_WEIGHT, class Source, class Of>
__device__ __forceinline__ Cut descend(const Source& from, u64 limit, uint32_t prefix, int bits, Of of, Shared& s, int wave, int lane) {
    Cut cut = {0, 0, 0, 0};
    if (bits < 32) cut.key = prefix >> bits << bits;
    while (bits > 0) {
        const int take = bits < kBits ? bits : kBits, shift = bits - take;
        clear_bins(1 << take, s, wave * 64 + lane);
        from.each(wave, lane, [&](int id, float x) {
            uint32_t k;
            u64 w;
            if (!of(id, x, k, w) || (bits < 32 && (k >> bits) != (cut.key >> bits))) return;
            const int bin = (k >> shift) & ((1 << take) - 1);
            atomicAdd(&s.h.count[bin], 1u);
            if (BY_WEIGHT && w) atomicAdd(&s.h.weight[bin], w);
        });
        __syncthreads();
        cut.key |= (uint32_t)pick_bin<BY_WEIGHT>(1 << take, limit, cut, s, wave, lane) << shift;
        bits = shift;
        __syncthreads();
    }
    return cut;
}

// A sum of weights, and a number of tokens at the edge, of which the first
// `tied` of the row weigh `each`.
struct Sum {
    u64 weight, ties;
};
struct Tied {
    u64 tied, each;

    // the weight of a part behind `before` tokens at the edge
    __device__ __forceinline__ u64 weight(const Sum& part, u64 before) const {
        const u64 upto = before + part.ties;
        return part.weight + ((upto < tied ? upto : tied) - (before < tied ? before : tied)) * each;
    }
};

// The first id with which the weight of what m.one(id, x, sum) adds up over the
// row passes `target`, which all of it does; target = of(the weight of all).
// m.group(g, v, sum) adds a group.
template <class E, class M, class Of>
__device__ __forceinline__ int locate(const Row<E>& row, const M& m, const Tied& tied, Of of, u64* total, Shared& s, int wave,
                                      int lane) {
    int g0 = 0, g1 = row.groups;
    u64 before = 0, ties = 0, target = 0;                  // weight and ties before group g0
    bool whole = true;
    do {
        // all waves, a part each; the part in which the target lies goes on
        const int per = (g1 - g0 + kWaves - 1) / kWaves;
        const int from = g0 + wave * per < g1 ? g0 + wave * per : g1, to = from + per < g1 ? from + per : g1;
        Sum sum = {0, 0};
        row.template groups_of<2>(from, to, lane, [&](int g, const u32x4& v) { m.group(g, v, sum); });
        sum.weight = wave_add_u64(sum.weight);
        sum.ties = wave_add_u64(sum.ties);
        if (lane == 0) {
            s.wave[0][wave] = sum.weight;
            s.wave[1][wave] = sum.ties;
        }
        __syncthreads();
        if (whole) {
            Sum all = {0, 0};
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                all.weight += s.wave[0][i];
                all.ties += s.wave[1][i];
            }
            *total = tied.weight(all, 0);
            target = of(*total);
            whole = false;
        }
        u64 upto = before, upto_ties = ties;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kWaves - 1; ++i) {
            const Sum part = {s.wave[0][i], s.wave[1][i]};
            upto += tied.weight(part, upto_ties);
            upto_ties += part.ties;
            if (upto <= target) {
                at = i + 1;
                before = upto;
                ties = upto_ties;
            }
        }
        const int n0 = g0 + at * per < g1 ? g0 + at * per : g1;
        g1 = n0 + per < g1 ? n0 + per : g1;
        g0 = n0;
        __syncthreads();
    } while (g1 - g0 > 4 * kThreads);
    // a thread a run of up to four groups
    const int per = (g1 - g0 + kThreads - 1) / kThreads, mine = g0 + (wave * 64 + lane) * per;
    Sum sum = {0, 0};
    for (int i = 0; i < per; ++i)
        if (mine + i < g1) m.group(mine + i, row.load(mine + i), sum);
    const u64 upto = wave_prefix_u64(sum.weight, lane), upto_ties = wave_prefix_u64(sum.ties, lane);
    if (lane == 63) {
        s.wave[0][wave] = upto;
        s.wave[1][wave] = upto_ties;
    }
    if (wave == 0 && lane == 0) s.found[0] = ~0ull;
    __syncthreads();
    Sum part = {upto - sum.weight, upto_ties - sum.ties};  // before this thread's run
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i) {
        part.weight += i < wave ? s.wave[0][i] : 0;
        part.ties += i < wave ? s.wave[1][i] : 0;
    }
    const u64 sofar = before + tied.weight(part, ties);
    ties += part.ties;
    if (sofar <= target && sofar + tied.weight(sum, ties) > target) {
        int found = -1;
        Sum run = {0, 0};
        for (int i = 0; i < per; ++i) {
            if (mine + i >= g1) break;
            const u32x4 v = row.load(mine + i);
#pragma unroll
            for (int e = 0; e < Row<E>::kEach; ++e) {
                const int id = (mine + i) * Row<E>::kEach - row.before + e;
                const float x = Row<E>::at(v, e);
                m.one(id, x == x ? x : -INFINITY, run);
                if (found < 0 && sofar + tied.weight(run, ties) > target) found = id;
            }
        }
        s.found[0] = (u64)found;
    }
    __syncthreads();
    return (int)s.found[0];
}

// Of a weight of id and logit.
template <class E, class F>
struct Each {
    const Row<E>& row;
    F f;

    __device__ __forceinline__ void one(int id, float x, Sum& sum) const { sum.weight += f(id, x); }
    __device__ __forceinline__ void group(int g, const u32x4& v, Sum& sum) const {
#pragma unroll
        for (int e = 0; e < Row<E>::kEach; ++e) {
            const float x = Row<E>::at(v, e);
            sum.weight += f(g * Row<E>::kEach - row.before + e, x == x ? x : -INFINITY);
        }
    }
};
template <class E, class F>
__device__ __forceinline__ Each<E, F> each_of(const Row<E>& row, F f) { return {row, f}; }

// What a request asks for, and the row's own measures.
struct Ask {
    int top_k;                     // 0: off
    float top_p;                   // >= 1: off
    u64 least;                     // weight that min_p asks for (0: off)
    double u;
    int first;                     // the largest logit's token, which always stays
    int id_bits;
    Weights weights;
};

__device__ __forceinline__ u64 limit_of(float top_p, u64 total) {
    const double part = ceil((double)top_p * (double)total);
    const u64 limit = part >= 1 ? (u64)part : 1;
    return limit < total ? limit : total;
}
__device__ __forceinline__ u64 target_of(double u, u64 total) {
    const double t = u * (double)total;
    return t >= 1 ? (t < (double)total ? (u64)t : total - 1) : 0;
}

// What stays: all tokens above `value`, and those at it up to id `last`.
struct Edge {
    float value;
    int last;
};

// The edge of top_k and top_p among the tokens of `from`, which hold everything
// that top_k leaves, or, without it, everything at the edge of top_p and what is
// above it but for tokens that weigh `above`, of all that weigh `total`.  Their
// keys have the bits of `prefix` from `bits` on.
template <class E, class Source>
__device__ __forceinline__ Edge find_edge(const Source& from, const Ask& ask, int count, u64 total, u64 above, uint32_t prefix, int bits,
                          Shared& s, int wave, int lane) {
    // keys of a 16-bit type are told apart by their upper half
    constexpr int kLow = sizeof(E) == 2 ? 16 : 0;
    const auto by_logit = [&](int, float x, uint32_t& k, u64& w) {
        if (x == -INFINITY) return false;
        k = key_of(x) >> kLow;
        return true;
    };
    const auto full = [&](uint32_t k) { return sizeof(E) == 2 ? (k & 0x8000u ? k << 16 : k << 16 | 0xFFFFu) : k; };
    bits = bits > kLow ? bits - kLow : 1;
    prefix >>= kLow;
    Edge edge = {-INFINITY, INT32_MAX};
    u64 tied = 0;
    bool part = false;                                     // only `tied` of the tokens at the edge stay
    if (ask.top_k > 0 && count > ask.top_k) {
        const Cut c = descend<false>(from, (u64)ask.top_k, prefix, bits, by_logit, s, wave, lane);
        edge.value = value_of(full(c.key));
        tied = (u64)ask.top_k - c.count;
        part = tied < c.ties;
    }
    if (ask.top_p < 1) {
        if (ask.top_k > 0) {                               // of what top_k leaves
            u64 sum = 0;
            from.each(wave, lane, [&](int, float x) {
                const u64 w = ask.weights(x);
                sum += x > edge.value || (x == edge.value && !part) ? w : 0;
            });
            total = block_add(sum, s, wave, lane);
            if (part) total += tied * ask.weights(edge.value);
        }
        const u64 limit = limit_of(ask.top_p, total) - above;
        const Cut c = descend<true>(from, limit, prefix, bits, [&](int id, float x, uint32_t& k, u64& w) {
            w = ask.weights(x);
            return by_logit(id, x, k, w);
        }, s, wave, lane);
        const float value = value_of(full(c.key));
        const u64 w = ask.weights(value), need = w ? (limit - c.weight + w - 1) / w : 0;
        if (value == edge.value && part) {
            tied = need < tied ? need : tied;
        } else {
            tied = need < c.ties ? need : c.ties;
            part = tied < c.ties;
        }
        edge.value = value;
    }
    if (part) {
        const Cut c = descend<false>(from, tied, 0, ask.id_bits, [&](int id, float x, uint32_t& k, u64&) {
            k = ((1u << ask.id_bits) - 1) - (uint32_t)id;  // the lowest ids on top
            return x == edge.value;
        }, s, wave, lane);
        edge.last = (int)(((1u << ask.id_bits) - 1) - c.key);
    }
    return edge;
}

__device__ __forceinline__ u64 kept_weight(const Ask& ask, const Edge& edge, int id, float x) {
    const u64 w = ask.weights(x);
    const bool stays = (x > edge.value || (x == edge.value && id <= edge.last)) && (w >= ask.least || id == ask.first);
    return stays ? w : 0;
}

// The token drawn from the list, which holds all that stay.
__device__ __forceinline__ int draw_listed(const List& list, const Ask& ask, const Edge& edge, u64* total, Shared& s, int wave, int lane) {
    u64 sum = 0;
    list.each(wave, lane, [&](int id, float x) { sum += kept_weight(ask, edge, id, x); });
    *total = block_add(sum, s, wave, lane);
    if (*total == 0) return ask.first;
    const Cut c = descend<true>(list, target_of(ask.u, *total) + 1, 0, ask.id_bits, [&](int id, float x, uint32_t& k, u64& w) {
        w = kept_weight(ask, edge, id, x);
        k = ((1u << ask.id_bits) - 1) - (uint32_t)id;
        return w > 0;
    }, s, wave, lane);
    return (int)(((1u << ask.id_bits) - 1) - c.key);
}

// The same as find_edge and draw_listed, from a short list that holds all that
// stays: every pair of its tokens is compared, two threads a token.
__device__ __forceinline__ int draw_short(const List& list, const Ask& ask, u64* total, Shared& s, int wave, int lane) {
    constexpr int kParts = kThreads / kShort;
    const int tid = wave * 64 + lane, i = tid / kParts, part = tid % kParts;
    const bool mine = i < list.n;
    const float x = mine ? s.h.list[i] : -INFINITY;
    const int id = mine ? s.h.ids[i] : INT32_MAX;
    const u64 w = mine ? ask.weights(x) : 0;
    if (mine && part == 0) s.h.weight[i] = w;
    __syncthreads();
    // those before it in the order: their number and weight
    uint32_t rank = 0;
    u64 before = 0;
    for (int j = part; j < list.n; j += kParts) {
        const float y = s.h.list[j];
        const bool first = y > x || (y == x && s.h.ids[j] < id);
        rank += first;
        before += first ? s.h.weight[j] : 0;
    }
#pragma unroll
    for (int d = 1; d < kParts; d <<= 1) {
        rank += __shfl_xor((int)rank, d);
        before += (u64)(uint32_t)__shfl_xor((int)(uint32_t)before, d) | (u64)(uint32_t)__shfl_xor((int)(uint32_t)(before >> 32), d) << 32;
    }
    bool stays = mine && (ask.top_k == 0 || rank < (uint32_t)ask.top_k);
    if (ask.top_p < 1) {
        const u64 all = block_add(stays && part == 0 ? w : 0, s, wave, lane);
        stays = stays && before < limit_of(ask.top_p, all);
    }
    stays = stays && (w >= ask.least || id == ask.first);
    const u64 kept = stays ? w : 0;
    *total = block_add(part == 0 ? kept : 0, s, wave, lane);
    if (*total == 0) return ask.first;
    if (mine && part == 0) s.h.weight[i] = kept;
    __syncthreads();
    // those before it by id
    u64 upto = 0;
    for (int j = part; j < list.n; j += kParts) upto += s.h.ids[j] < id ? s.h.weight[j] : 0;
#pragma unroll
    for (int d = 1; d < kParts; d <<= 1)
        upto += (u64)(uint32_t)__shfl_xor((int)(uint32_t)upto, d) | (u64)(uint32_t)__shfl_xor((int)(uint32_t)(upto >> 32), d) << 32;
    const u64 target = target_of(ask.u, *total);
    if (part == 0 && upto <= target && target < upto + kept) s.found[0] = (u64)id;
    __syncthreads();
    return (int)s.found[0];
}

typedef __attribute__((address_space(3))) char* Lds;

// Weights of 16-bit logits by their bits: a read of LDS in place of some thirty
// instructions.
struct ByValue {
    Shared& s;
    int base;                      // bits of the smallest magnitude there

    // exponents up to one past those of the largest logit and of the smallest that
    // weighs anything
    __device__ __forceinline__ ByValue(Shared& s_, float top, float low) : s(s_) {
        const int m = (int)(__float_as_uint(fmaxf(fabsf(top), fabsf(low))) >> 23);     // (inf: 255)
        const int first = m + 2 - kBinades;
        base = (first < 0 ? 0 : (first > 256 - kBinades ? 256 - kBinades : first)) << 7;
    }
    __device__ __forceinline__ float value(int i, int negative) const {
        return __uint_as_float((uint32_t)(base + i + (negative ? 0x8000 : 0)) << 16);
    }
    // Places in the arrays of a group's eight logits, two at a time.  NaN,
    // infinities and others past the end go to the last one, which weighs nothing;
    // whether there are any, and whether there are tiny ones.
    __device__ __forceinline__ void places(const u32x4& v, uint32_t (&at)[8], bool& past, bool& tiny) const {
        typedef short i16x2 __attribute__((ext_vector_type(2)));
        constexpr short kLast = kMagnitudes - 1;
        const i16x2 from = {(short)base, (short)base}, last = {kLast, kLast}, none = {0, 0};
        i16x2 least = none, most = none;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const i16x2 i = __builtin_bit_cast(i16x2, v[d] & 0x7FFF7FFFu) - from;
            least = __builtin_elementwise_min(least, i);
            most = __builtin_elementwise_max(most, i);
            const i16x2 in = __builtin_elementwise_max(__builtin_elementwise_min(i, last), none);
            // (both halves at once: a sum stays below 2^16)
            const uint32_t p = __umul24(v[d] >> 15 & 0x10001u, kMagnitudes) + __builtin_bit_cast(uint32_t, in);
            at[2 * d] = p & 0xFFFF;
            at[2 * d + 1] = p >> 16;
        }
        past = most[0] >= kLast || most[1] >= kLast;
        tiny = least[0] < 0 || least[1] < 0;
    }
    __device__ __forceinline__ bool is_tiny(float x) const { return (int)((__float_as_uint(x) >> 16) & 0x7FFF) < base; }
    __device__ __forceinline__ u64 weight(float x) const { // not of tiny ones
        const int i = (int)((__float_as_uint(x) >> 16) & 0x7FFF) - base;
        return s.v.weight[(i < kMagnitudes - 1 ? i : kMagnitudes - 1) + ((__float_as_int(x) >> 31) & kMagnitudes)];
    }
    // `ties`: those at the edge are counted apart, and weigh nothing here
    __device__ __forceinline__ void fill(const Ask& ask, const Edge& edge, bool ties, int tid) const {
        for (int i = tid; i < kMagnitudes; i += kThreads)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float x = value(i, n);
                const bool stays = i < kMagnitudes - 1 && x <= (float)ask.weights.top && (ties ? x > edge.value : x >= edge.value);
                const u64 w = stays ? ask.weights(x) : 0;
                s.v.weight[n * kMagnitudes + i] = w >= ask.least ? w : 0;
            }
        __syncthreads();
    }
    // the order's beginning that reaches `limit` in number (or weight): its last
    // value's, false where that is a tiny one
    template <bool BY_WEIGHT>
    __device__ __forceinline__ bool cut(u64 limit, float& x, Cut& c, int wave, int lane) const {
        // from the top: positive values, the tiny ones, negative values; so many a thread
        constexpr int kEach = (2 * kMagnitudes + kThreads) / kThreads;
        const int q0 = (wave * 64 + lane) * kEach;
        const auto bin = [&](int q, u64& n, u64& w) {
            n = w = 0;
            if (q == kMagnitudes) {
                n = s.tiny_count;
                w = s.tiny_weight;
            } else if (q <= 2 * kMagnitudes) {
                const int at = q < kMagnitudes ? kMagnitudes - 1 - q : q - 1;
                n = s.v.count[at];
                w = n * s.v.weight[at];
            }
        };
        u64 n = 0, w = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            u64 ni, wi;
            bin(q0 + i, ni, wi);
            n += ni;
            w += wi;
        }
        const u64 np = wave_prefix_u64(n, lane), wp = wave_prefix_u64(w, lane);
        if (lane == 63) {
            s.wave[0][wave] = np;
            s.wave[1][wave] = wp;
        }
        if (wave == 0 && lane == 0) s.found[0] = (u64)kMagnitudes;
        __syncthreads();
        u64 nx = np - n, wx = wp - w;
#pragma unroll
        for (int i = 0; i < kWaves - 1; ++i) {
            nx += i < wave ? s.wave[0][i] : 0;
            wx += i < wave ? s.wave[1][i] : 0;
        }
        for (int i = 0; i < kEach; ++i) {
            u64 ni, wi;
            bin(q0 + i, ni, wi);
            const u64 m = BY_WEIGHT ? wx : nx;
            if (m < limit && m + (BY_WEIGHT ? wi : ni) >= limit) {
                s.found[0] = (u64)(q0 + i);
                s.found[1] = nx;
                s.found[2] = wx;
                s.found[3] = ni;
            }
            nx += ni;
            wx += wi;
        }
        __syncthreads();
        const int q = (int)s.found[0];
        c.count = (uint32_t)s.found[1];
        c.weight = s.found[2];
        c.ties = (uint32_t)s.found[3];
        x = q < kMagnitudes ? value(kMagnitudes - 1 - q, 0) : value(q - kMagnitudes - 1, 1);
        __syncthreads();
        return q != kMagnitudes;
    }
};

// What is kept of a row, by the weights that fill() has left of the values.
template <class E>
struct KeptByValue {
    const Row<E>& row;
    const ByValue& by;
    const Ask& ask;
    const Edge& edge;
    bool ties;

    __device__ __forceinline__ void one(int id, float x, Sum& sum) const {
        if (ties && x == edge.value) ++sum.ties;
        else if (by.is_tiny(x)) sum.weight += kept_weight(ask, edge, id, x);
        else if (x != edge.value || id <= edge.last) sum.weight += by.weight(x);
    }
    // the reads of LDS side by side; tiny logits, usually few, one by one
    __device__ __forceinline__ void group(int g, const u32x4& v, Sum& sum) const {
        uint32_t at[8];
        u64 w[8];
        bool past, tiny;
        by.places(v, at, past, tiny);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = by.s.v.weight[at[e]];
        if (ties) {
            uint32_t n = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) n += Row<E>::at(v, e) == edge.value;
            sum.ties += n;
        }
        if (__any(tiny) || edge.last < INT32_MAX) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = Row<E>::at(v, e);
                const int id = g * 8 - row.before + e;
                if (x == edge.value && id > edge.last) w[e] = 0;
                if (by.is_tiny(x)) w[e] = ties && x == edge.value ? 0 : kept_weight(ask, edge, id, x);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.weight += w[e];
    }
};

// Counts every value of the row.  Tiny logits (magnitudes below the 22 binades:
// exact zeros at ordinary temperatures) take three atomics on the same words: 512
// rows of 151936 bf16 with top_p 137 us, 244 where 1% of the logits are 0, 1410
// where half are, 2430 where 99% are (one row 62, 140, 554 and 1590).
template <class E>
__device__ __forceinline__ void count_values(const Row<E>& row, const ByValue& by, const Ask& ask, int wave, int lane) {
    const int tid = wave * 64 + lane, per = (row.groups + kWaves - 1) / kWaves;
    const int g0 = wave * per < row.groups ? wave * per : row.groups, g1 = g0 + per < row.groups ? g0 + per : row.groups;
    for (int i = tid; i < 2 * kMagnitudes; i += kThreads) by.s.v.count[i] = 0;
    if (tid == 0) {
        by.s.tiny_weight = 0;
        by.s.tiny_count = 0;
    }
    __syncthreads();
    row.template groups_of<2>(g0, g1, lane, [&](int, const u32x4& v) {
        uint32_t at[8];
        bool past, tiny;
        by.places(v, at, past, tiny);
        if (__any(tiny)) {
            // (counted at the smallest magnitude, too, and taken out there)
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                const uint32_t word = e < 2 ? v[0] : (e < 4 ? v[1] : (e < 6 ? v[2] : v[3]));
                const float x = __uint_as_float(e & 1 ? word & 0xFFFF0000u : word << 16);
                if (!by.is_tiny(x)) continue;
                atomicAdd(&by.s.tiny_count, 1u);
                atomicAdd(&by.s.tiny_weight, ask.weights(x));
                atomicSub(&by.s.v.count[(word >> (16 * (e & 1)) & 0x8000) ? kMagnitudes : 0], 1u);
            }
        }
        if (__any(past)) {
            // what weighs nothing is not counted: half of a row may be -inf, all at one place
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at[e] != kMagnitudes - 1 && at[e] != 2 * kMagnitudes - 1) atomicAdd(&by.s.v.count[at[e]], 1u);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) atomicAdd(&by.s.v.count[at[e]], 1u);
        }
    });
    __syncthreads();
    // -0 is 0 (where magnitudes begin at 0; otherwise both are tiny)
    if (by.base == 0 && tid == 0) {
        by.s.v.count[0] += by.s.v.count[kMagnitudes];
        by.s.v.count[kMagnitudes] = 0;
    }
    __syncthreads();
}

// The edge of top_k and top_p by the counted values; false where it is not to be
// had so.  `tied` of the tokens at it stay, if `part`.
__device__ __forceinline__ bool edge_by_value(const ByValue& by, const Ask& ask, Edge& edge, u64& tied, bool& part, Shared& s,
                                              int wave, int lane) {
    Cut c;
    float x;
    u64 total = 0, n = 0;
    for (int i = wave * 64 + lane; i < 2 * kMagnitudes; i += kThreads) {
        total += s.v.count[i] * s.v.weight[i];
        n += s.v.count[i];
    }
    n = block_add(n, s, wave, lane) + by.s.tiny_count;
    total = block_add(total, s, wave, lane) + by.s.tiny_weight;
    if (ask.top_k > 0 && n > (u64)ask.top_k) {             // (what is not counted weighs nothing)
        if (!by.cut<false>((u64)ask.top_k, x, c, wave, lane)) return false;
        edge.value = x;
        tied = (u64)ask.top_k - c.count;
        part = tied < c.ties;
        total = c.weight + tied * ask.weights(x);
    }
    if (ask.top_p < 1) {
        const u64 limit = limit_of(ask.top_p, total);
        if (!by.cut<true>(limit, x, c, wave, lane)) return false;
        const u64 w = ask.weights(x), need = w ? (limit - c.weight + w - 1) / w : 0;
        if (x == edge.value && part) {
            tied = need < tied ? need : tied;
        } else {
            tied = need < c.ties ? need : c.ties;
            part = tied < c.ties;
        }
        edge.value = x;
    }
    return true;
}

// All tokens for which wanted(x) into the list; whether they fit.  wanted sees
// every logit on the way, -inf and NaN among them.
template <class E, class F>
__device__ __forceinline__ bool make_list(const Row<E>& row, F wanted, Shared& s, int wave, int lane) {
    if (wave == 0 && lane == 0) s.listed = 0;
    __syncthreads();
    const int per = (row.groups + kWaves - 1) / kWaves, g0 = wave * per < row.groups ? wave * per : row.groups;
    row.template groups_of<4>(g0, g0 + per < row.groups ? g0 + per : row.groups, lane, [&](int g, const u32x4& v) {
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < Row<E>::kEach; ++e) mine |= wanted(Row<E>::at(v, e)) ? 1u << e : 0u;
        if (__any(mine != 0)) {
            uint32_t all = 0, to[Row<E>::kEach];
#pragma unroll
            for (int e = 0; e < Row<E>::kEach; ++e) {
                const u64 hit = __ballot(mine >> e & 1);
                to[e] = all + __builtin_amdgcn_mbcnt_hi((uint32_t)(hit >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)hit, 0));
                all += (uint32_t)__popcll(hit);
            }
            uint32_t at = 0;
            if (lane == 0) at = atomicAdd(&s.listed, all);
            at = (uint32_t)__builtin_amdgcn_readfirstlane((int)at);
#pragma unroll
            for (int e = 0; e < Row<E>::kEach; ++e)
                if ((mine >> e & 1) && at + to[e] < kList) {
                    s.h.list[at + to[e]] = Row<E>::at(v, e);
                    s.h.ids[at + to[e]] = g * Row<E>::kEach - row.before + e;
                }
        }
    });
    __syncthreads();
    return s.listed <= kList;
}

// Each thread's two largest logits (of different groups).
struct Largest {
    float mine, second;

    template <class F>
    __device__ __forceinline__ void each(int, int, F f) const {
        f(0, mine);
        f(0, second);
    }
};

template <class E>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(SampleArgs a, int shift) {
    // 16-bit logits have few values: each one's weight is made once
    constexpr bool kValues = sizeof(E) == 2;
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t at = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (at >= (int64_t)a.B * a.rows) return;
    const int b = (int)(at / a.rows), r = (int)(at - (int64_t)b * a.rows);
    if (r >= a.lead && a.n_nodes && r - a.lead >= a.n_nodes[b]) return;    // (any number: a sum could pass 32 bits)
    const Row<E> row(a.logits, at, a.V);
    if (tid < kTable) s.table[tid] = ldexp(exp2((double)tid / kTable), shift);

    // the largest logit and its first id: each lane's largest, and where it was met first
    const int per = (row.groups + kWaves - 1) / kWaves, g0 = wave * per < row.groups ? wave * per : row.groups;
    float mine = -INFINITY, second = -INFINITY;
    int where = 0;
    row.template groups_of<4>(g0, g0 + per < row.groups ? g0 + per : row.groups, lane, [&](int g, const u32x4& v) {
        // (a sum's NaN is a quiet one, of which fmaxf takes the number beside it; of a signalling one it would not)
        float x = -INFINITY;
#pragma unroll
        for (int e = 0; e < Row<E>::kEach; ++e) x = fmaxf(x, Row<E>::at(v, e) + 0.0f);
        second = fmaxf(second, fminf(mine, x));
        where = x > mine ? g : where;
        mine = x > mine ? x : mine;
    });
    const float wave_top = wave_max_f32(mine);
    if (lane == 0) s.wave[0][wave] = key_of(wave_top);
    if (tid == 0) s.found[0] = (u64)a.V;
    __syncthreads();
    u64 top_key = 0;
    for (int i = 0; i < kWaves; ++i) top_key = s.wave[0][i] > top_key ? s.wave[0][i] : top_key;
    const float top = value_of((uint32_t)top_key);
    const float temperature = a.temperature ? a.temperature[b] : 1.0f;
    if (top == -INFINITY) {
        if (tid == 0) {
            a.tokens[at] = -1;
            if (a.logp) a.logp[at] = -INFINITY;
        }
        return;
    }
    if (mine == top) {
        const u32x4 v = row.load(where);
        int e0 = 0;
#pragma unroll
        for (int e = Row<E>::kEach - 1; e >= 0; --e) e0 = Row<E>::at(v, e) == top ? e : e0;
        atomicMin(&s.found[0], (u64)(where * (int64_t)Row<E>::kEach - row.before + e0));
    }
    __syncthreads();
    Ask ask;
    ask.first = (int)s.found[0];
    if (!(temperature > 0)) {
        if (tid == 0) {
            a.tokens[at] = ask.first;
            if (a.logp) a.logp[at] = 0.0f;
        }
        return;
    }
    const int top_k = a.top_k ? a.top_k[b] : 0;
    const float min_p = a.min_p ? a.min_p[b] : 0.0f;
    ask.top_k = top_k > 0 && top_k < a.V ? top_k : 0;
    ask.top_p = a.top_p ? a.top_p[b] : 1.0f;
    ask.least = min_p > 0 ? (u64)ceil(ldexp((double)(min_p < 2.0f ? min_p : 2.0f), shift)) : 0;
    ask.u = a.u[at];
    ask.id_bits = 32 - __clz(a.V - 1 > 0 ? a.V - 1 : 1);
    ask.weights = {(double)top, kTable * 1.4426950408889634074 / (double)temperature, -(double)kTable * (shift + 2), (Table)s.table};
    const bool by_p = ask.top_p < 1;

    Edge edge = {-INFINITY, INT32_MAX};
    u64 total = 0, all = 0, above = 0;
    int token = -1, n = 0;
    // what the list holds: nothing, all that stays, or the tokens around the edge
    enum { kNothing, kAll, kEdge } holds = kNothing;
    uint32_t low = 0;                                      // the smallest key there
    bool edged = false, part = false;
    u64 tied = 0;
    if constexpr (kValues) {
        if (ask.top_k > kMostK || (by_p && ask.top_k == 0)) {
            const ByValue by(s, top, top - (shift + 2) * 0.6931472f * temperature);
            Ask any = ask;
            any.least = 0;
            by.fill(any, edge, false, tid);
            count_values(row, by, ask, wave, lane);
            edged = edge_by_value(by, ask, edge, tied, part, s, wave, lane);
            if (!edged) {
                edge = {-INFINITY, INT32_MAX};
                part = false;
            }
        }
    }
    if (edged) {
        // the row itself, below
    } else if (ask.top_k <= kMostK && ((by_p && !kValues) || ask.top_k > 0)) {
        // the logit that j threads' largest reach (its upper 22 bits)
        const u64 j = ask.top_k > 0 ? ask.top_k : kForP;
        const Largest largest{mine, second};
        float limit = -FLT_MAX;
        if (block_add((u64)(mine > -INFINITY) + (second > -INFINITY), s, wave, lane) >= j) {
            const Cut c = descend<false>(largest, j, 0, 22, [&](int, float x, uint32_t& k, u64&) {
                k = key_of(x) >> 10;
                return x > -INFINITY;
            }, s, wave, lane);
            limit = value_of(c.key << 10);
        }
        low = key_of(limit);
        if (ask.top_k > 0) {
            if (make_list(row, [&](float x) { return x >= limit; }, s, wave, lane)) holds = kAll;
            n = (int)s.listed;
        } else {
            // bins over the logits that weigh anything, the largest in the last
            const float width = (kBins - 1) / ((shift + 1) * 0.6931472f * temperature);
            const auto bin_of = [&](float x) { return kBins - 1 - (int)fminf((top - x) * width, (float)(kBins - 1)); };
            clear_bins(kBins, s, tid);
            const bool fits = make_list(row, [&](float x) {
                const u64 w = ask.weights(x);
                if (w) atomicAdd(&s.h.weight[bin_of(x)], w);
                return x >= limit;
            }, s, wave, lane);
            n = (int)s.listed;
            for (int i = tid; i < kBins; i += kThreads) all += s.h.weight[i];
            all = block_add(all, s, wave, lane);
            Cut c = {0, 0, 0, 0};
            const int bin = pick_bin<true>(kBins, limit_of(ask.top_p, all), c, s, wave, lane);
            __syncthreads();
            if (fits && bin_of(limit) < bin) {             // the list holds the cut and all above
                holds = kAll;
            } else if (make_list(row, [&](float x) { return bin_of(x) == bin && x > -INFINITY && ask.weights(x) > 0; }, s, wave, lane)) {
                holds = kEdge;
                n = (int)s.listed;
                above = c.weight;
                low = 0;
            }
        }
    } else if (!by_p && ask.top_k == 0 && ask.least > 0) {
        // what min_p leaves, weights that round up to it among them, and a little more
        // for the roundings of weights (below 2^-43 of them) and of this limit
        const double below = (double)temperature * (fmin(log(ldexp((double)ask.least - 0.5, -shift)), 0.0) - 1e-12);
        const float limit = fmaxf((float)((double)top + below - 1e-6 * (fabs((double)top) - below) - 1e-37), -FLT_MAX);
        if (make_list(row, [&](float x) { return x >= limit; }, s, wave, lane)) holds = kAll;
        n = (int)s.listed;
    }
    const List list{s, n};
    if (holds == kAll && n <= kShort && !(by_p && ask.top_k == 0)) {
        // (top_p alone goes by the weight of the whole row)
        token = draw_short(list, ask, &total, s, wave, lane);
    } else if (!edged && (by_p || ask.top_k > 0)) {
        if (holds != kNothing) {
            const int bits = 32 - __clz((low ^ (uint32_t)top_key) | 1);
            edge = find_edge<E>(list, ask, n, all, above, low, bits, s, wave, lane);
        } else {
            u64 there = 0;
            all = 0;
            row.each(wave, lane, [&](int, float x) {
                there += x != -INFINITY;
                all += ask.weights(x);
            });
            there = block_add(there, s, wave, lane);
            all = block_add(all, s, wave, lane);
            edge = find_edge<E>(row, ask, (int)there, all, 0, 0, 32, s, wave, lane);
        }
    }
    if (token >= 0) {
    } else if (holds == kAll) {
        token = draw_listed(list, ask, edge, &total, s, wave, lane);
    } else {
        const auto of = [&](u64 sum) { return target_of(ask.u, sum); };
        if constexpr (kValues) {
            const ByValue by(s, top, top - (shift + 2) * 0.6931472f * temperature);
            by.fill(ask, edge, part, tid);
            const u64 each = part ? ask.weights(edge.value) : 0;
            const Tied at_edge = {tied, each >= ask.least ? each : 0};
            // (min_p above 1: `first` alone)
            token = ask.least > 1ull << shift ? -1
                                              : locate(row, KeptByValue<E>{row, by, ask, edge, part}, at_edge, of, &total, s, wave, lane);
            if (ask.least > 1ull << shift) total = 1ull << shift;
        } else {
            token = locate(row, each_of(row, [&](int id, float x) { return kept_weight(ask, edge, id, x); }), Tied{0, 0}, of,
                           &total, s, wave, lane);
        }
    }
    if (tid == 0) {
        token = token < 0 || token >= a.V ? ask.first : token;
        a.tokens[at] = token;
        if (a.logp) {
            const float x = Row<E>::get(((const E*)a.logits)[at * a.V + token]);
            a.logp[at] = (float)(((double)x - (double)top) / (double)temperature - log(ldexp((double)total, -shift)));
        }
    }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t stream) {
    int n = 0;
    while ((1ll << n) < a.V) ++n;
    const int shift = 62 - n < 50 ? 62 - n : 50;
    // threads along x count in 32 bits, fewer than 2^23 rows: from 2^20 on they go on in y
    const unsigned rows = (unsigned)((int64_t)a.B * a.rows), x = rows < kMaxGridX ? rows : kMaxGridX;
    const dim3 grid(x, (rows + x - 1) / x);
    if (dtype == DT_DTYPE_BF16) sample_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(a, shift);
    else sample_kernel<uint32_t><<<grid, kThreads, 0, stream>>>(a, shift);
    return hipGetLastError();
}

}  // namespace dt
