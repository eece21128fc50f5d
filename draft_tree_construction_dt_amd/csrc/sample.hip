// dt_sample_rows: a token for every row of logits, drawn by a given random
// number among those that top-k, top-p and min-p leave.
//
// What stays is a beginning of the order (logit desc, id asc): all tokens above
// some logit, and the first few by id of those at it.  With the weights held as
// integers (w scaled by 2^shift, so that V of them fit 62 bits) every sum is
// exact, whatever its order and grouping: the cut can be narrowed digit by digit
// over the logits' bits with histograms in LDS, the drawn token part by part
// over the ids, and neither ever meets two sums that should agree and do not.
//
// A workgroup takes a row.
#include <math.h>

#include "pass.h"
#include "wave.h"

namespace dt {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;        // of a histogram: 11 bits of a logit at a time
constexpr int kDeep = 4;           // 16-byte loads of a lane in flight

// Bits whose order is that of the values (no NaN).
__device__ inline uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
__device__ inline float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// e^((x - top) / temperature) * 2^shift, rounded: 2^(j / 64) from a table times
// the series of 2^(f / 64), |f| <= 1/2, to the fourth power; the next term is
// below 2^-44.  In fp64: a sum over V weights is compared with u times the total,
// and errors of 2^-24 a weight would move the drawn token in one row of a
// thousand.
struct Weights {
    double top, rate;              // rate = 64 log2(e) / temperature
    double least;                  // below it a weight is 0
    int shift;
    const double* table;           // LDS, 2^(j / 64)

    __device__ u64 operator()(float x) const {
        const double t = ((double)x - top) * rate;
        if (!(t > least)) return 0;
        const double n = rint(t), g = (t - n) * (0.69314718055994530942 / 64);
        const int i = (int)n;
        const double p = 1 + g * (1 + g * (0.5 + g * (1.0 / 6 + g * (1.0 / 24))));
        const double w = ldexp(table[i & 63] * p, (i >> 6) + shift);       // at most 2^50
        return (u64)__double_as_longlong(w + 4503599627370496.0) & 0xFFFFFFFFFFFFFull;
    }
};

// One row in memory, in groups of 16 aligned bytes; a group may begin before the
// row or end behind it.
template <class E>
struct Row {
    static constexpr int kEach = 16 / sizeof(E);
    const E* base;                 // of group 0
    int before, V, groups;         // elements of group 0 that are not the row's

    __device__ Row(const void* logits, int64_t row, int V_) : V(V_) {
        const int64_t at = row * V_;
        before = (int)(at % kEach);
        base = (const E*)logits + (at - before);
        groups = (int)(((int64_t)before + V_ + kEach - 1) / kEach);
    }
    static __device__ float get(uint32_t bits) {
        return sizeof(E) == 2 ? __uint_as_float(bits << 16) : __uint_as_float(bits);
    }
    // f(id, x) for every element of groups g0 .. g1 - 1 by one wave; the waves'
    // lanes stay together (f may use the whole wave: what is not there comes
    // as id -1, x = -inf).  NaN come as -inf, too.
    template <class F>
    __device__ void scan(int g0, int g1, int lane, F f) const {
        for (int64_t first = g0; first < g1; first += kDeep * 64) {
            u32x4 v[kDeep];
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                const int64_t g = first + i * 64 + lane;
                v[i] = u32x4{0, 0, 0, 0};
                if (g >= g1) continue;
                const int64_t id = g * kEach - before;
                if (id >= 0 && id + kEach <= V) {
                    v[i] = *(const u32x4*)(base + g * kEach);
                } else {
                    for (int e = 0; e < kEach; ++e)
                        if (id + e >= 0 && id + e < V) {
                            const uint32_t b = base[g * kEach + e];
                            if constexpr (sizeof(E) == 2) v[i][e >> 1] |= b << (16 * (e & 1));
                            else v[i][e] = b;
                        }
                }
            }
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                const int64_t g = first + i * 64 + lane, id0 = g * kEach - before;
                if (first + i * 64 >= g1) break;
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const uint32_t b = sizeof(E) == 2 ? (v[i][e >> 1] >> (16 * (e & 1))) & 0xFFFF : v[i][e];
                    const bool there = g < g1 && id0 + e >= 0 && id0 + e < V;
                    const float x = get(b) + 0.0f;         // (-0 as 0: they are equal)
                    f(there ? (int)(id0 + e) : -1, there && x == x ? x : -INFINITY);
                }
            }
        }
    }
};

struct Shared {
    double table[64];
    uint32_t count[kBins];
    u64 weight[kBins];
    u64 wave[2][kWaves];
    u64 found[4];
};

__device__ inline u64 wave_add_u64(u64 v) {
#pragma unroll
    for (int s = 0; s < 4; ++s) v += dpp_step64(v, s);
    return (readlane64(v, 0) + readlane64(v, 16)) + (readlane64(v, 32) + readlane64(v, 48));
}
__device__ inline u64 wave_prefix_u64(u64 v, int lane) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const u64 o = (u64)(uint32_t)__shfl_up((int)(uint32_t)v, s) | (u64)(uint32_t)__shfl_up((int)(uint32_t)(v >> 32), s) << 32;
        if (lane >= s) v += o;
    }
    return v;
}

// Where the order's beginning ends: at logits of this key, above which lie
// `count` tokens of `weight` in all; `ties` tokens are at it.
struct Cut {
    uint32_t key;
    uint32_t count, ties;
    u64 weight;
};

// The first key, from the top, with which the tokens' number (or weight) reaches
// `limit`, which the whole row reaches.
template <class E, bool BY_WEIGHT>
__device__ Cut descend(const Row<E>& row, const Weights& weights, u64 limit, Shared& s, int wave, int lane) {
    const int tid = wave * 64 + lane, per = (row.groups + kWaves - 1) / kWaves;
    const int g0 = wave * per, g1 = g0 + per < row.groups ? g0 + per : row.groups;
    Cut cut = {0, 0, 0, 0};
    int above = 32;                                        // the bits at and above this are settled
    for (int level = 0; level < 3; ++level) {
        const int bits = level == 2 ? 10 : 11, shift = above - bits, bins = 1 << bits;
        for (int i = tid; i < kBins; i += kThreads) {
            s.count[i] = 0;
            s.weight[i] = 0;
        }
        __syncthreads();
        row.scan(g0, g1, lane, [&](int, float x) {
            if (x == -INFINITY) return;
            const uint32_t k = key_of(x);
            if (above < 32 && (k >> above) != (cut.key >> above)) return;
            const int bin = (k >> shift) & (bins - 1);
            atomicAdd(&s.count[bin], 1u);
            const u64 w = weights(x);
            if (w) atomicAdd(&s.weight[bin], w);
        });
        __syncthreads();
        // thread t's bins are the t-th pair from the top
        const int b0 = bins - 1 - 2 * tid, b1 = b0 - 1;
        const u64 c0 = b0 >= 0 ? s.count[b0] : 0, c1 = b1 >= 0 ? s.count[b1] : 0;
        const u64 w0 = b0 >= 0 ? s.weight[b0] : 0, w1 = b1 >= 0 ? s.weight[b1] : 0;
        const u64 cp = wave_prefix_u64(c0 + c1, lane), wp = wave_prefix_u64(w0 + w1, lane);
        if (lane == 63) {
            s.wave[0][wave] = cp;
            s.wave[1][wave] = wp;
        }
        __syncthreads();
        u64 cb = cut.count, wb = cut.weight;
        for (int i = 0; i < wave; ++i) {
            cb += s.wave[0][i];
            wb += s.wave[1][i];
        }
        const u64 cx = cb + cp - c0 - c1, wx = wb + wp - w0 - w1;      // before this thread's bins
        const u64 m0 = BY_WEIGHT ? wx : cx, m1 = BY_WEIGHT ? wx + w0 : cx + c0, m2 = BY_WEIGHT ? wx + w0 + w1 : cx + c0 + c1;
        const bool in0 = m0 < limit && m1 >= limit, in1 = m1 < limit && m2 >= limit;
        if (in0 || in1) {
            s.found[0] = (u64)(in0 ? b0 : b1);
            s.found[1] = in0 ? cx : cx + c0;
            s.found[2] = in0 ? wx : wx + w0;
            s.found[3] = in0 ? c0 : c1;
        }
        __syncthreads();
        cut.key |= (uint32_t)s.found[0] << shift;
        cut.count = (uint32_t)s.found[1];
        cut.weight = s.found[2];
        cut.ties = (uint32_t)s.found[3];
        above = shift;
        __syncthreads();
    }
    return cut;
}

// The first id with which the sum of m(id, x) passes `target`, which the whole
// row does, and the total; target = of(total).
template <class E, class M, class Of>
__device__ int locate(const Row<E>& row, M m, Of of, u64* total, Shared& s, int wave, int lane) {
    int g0 = 0, g1 = row.groups;
    u64 before = 0, target = 0;
    for (int level = 0; level < 3; ++level) {
        // all waves, a part each; the part in which the target lies goes on
        const int per = (g1 - g0 + kWaves - 1) / kWaves;
        const int from = g0 + wave * per < g1 ? g0 + wave * per : g1, to = from + per < g1 ? from + per : g1;
        u64 sum = 0;
        row.scan(from, to, lane, [&](int id, float x) { sum += m(id, x); });
        sum = wave_add_u64(sum);
        if (lane == 0) s.wave[0][wave] = sum;
        __syncthreads();
        if (level == 0) {
            u64 all = 0;
            for (int i = 0; i < kWaves; ++i) all += s.wave[0][i];
            *total = all;
            target = of(all);
        }
        int at = 0;
        for (; at < kWaves - 1 && before + s.wave[0][at] <= target; ++at) before += s.wave[0][at];
        const int n0 = g0 + at * per < g1 ? g0 + at * per : g1;
        g1 = n0 + per < g1 ? n0 + per : g1;
        g0 = n0;
        __syncthreads();
    }
    // what is left: 1/4096 of the row, element by element
    int found = -1;
    for (int g = g0; g < g1 && found < 0; g += 64) {
        // lanes hold groups: a group's sum first
        u64 sum = 0;
        row.scan(g, g + 64 < g1 ? g + 64 : g1, lane, [&](int id, float x) { sum += m(id, x); });
        const u64 upto = wave_prefix_u64(sum, lane);
        const u64 hit = __ballot(before + upto > target);
        if (!hit) {
            before += readlane64(upto, 63);
            continue;
        }
        const int l = __builtin_ctzll(hit);
        u64 sofar = before + readlane64(upto, l) - readlane64(sum, l);
        row.scan(g + l, g + l + 1, lane, [&](int id, float x) {
            const u64 w = m(id, x);                        // (lane 0's: the others have no group)
            if (lane == 0 && found < 0 && id >= 0) {
                sofar += w;
                if (sofar > target) found = id;
            }
        });
        found = __builtin_amdgcn_readlane(found, 0);
    }
    return found;
}

template <class E>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a, int shift) {
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t at = blockIdx.x;
    const int b = (int)(at / a.rows), r = (int)(at - (int64_t)b * a.rows);
    if (r >= a.lead && a.n_nodes && r >= a.lead + a.n_nodes[b]) return;
    const Row<E> row(a.logits, at, a.V);
    const int per = (row.groups + kWaves - 1) / kWaves;
    if (tid < 64) s.table[tid] = exp2(tid / 64.0);

    // the largest logit and its first id
    u64 best = 0;
    row.scan(wave * per, (wave + 1) * per < row.groups ? (wave + 1) * per : row.groups, lane, [&](int id, float x) {
        if (x == -INFINITY) return;
        const u64 k = (u64)key_of(x) << 32 | (uint32_t)~id;
        best = k > best ? k : best;
    });
    best = wave_max_u64(best);
    if (lane == 0) s.wave[0][wave] = best;
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) best = s.wave[0][i] > best ? s.wave[0][i] : best;
    __syncthreads();
    const float temperature = a.temperature ? a.temperature[b] : 1.0f;
    if (best == 0 || !(temperature > 0)) {
        if (tid == 0) {
            a.tokens[at] = best == 0 ? -1 : (int)~(uint32_t)best;
            if (a.logp) a.logp[at] = best == 0 ? -INFINITY : 0.0f;
        }
        return;
    }
    const int first = (int)~(uint32_t)best;
    Weights weights;
    weights.top = (double)value_of((uint32_t)(best >> 32));
    weights.rate = 64 * 1.4426950408889634074 / (double)temperature;
    weights.shift = shift;
    weights.least = -64.0 * (shift + 2);
    weights.table = s.table;

    // the cut: all tokens above `key`, and those at it up to `last`
    const int top_k = a.top_k ? a.top_k[b] : 0;
    const float top_p = a.top_p ? a.top_p[b] : 1.0f, min_p = a.min_p ? a.min_p[b] : 0.0f;
    const u64 least = min_p > 0 ? (u64)ceil(ldexp((double)(min_p < 2.0f ? min_p : 2.0f), shift)) : 0;
    uint32_t key = 0;                                      // (below every finite logit's)
    int last = a.V;
    bool cut_ties = false;
    u64 tied = 0;
    u64 total = 0;
    if (top_k > 0 && top_k < a.V) {
        u64 there = 0;
        // fewer finite logits than that: nothing to cut
        row.scan(wave * per, (wave + 1) * per < row.groups ? (wave + 1) * per : row.groups, lane,
                 [&](int, float x) { there += x != -INFINITY; });
        there = wave_add_u64(there);
        if (lane == 0) s.wave[0][wave] = there;
        __syncthreads();
        there = 0;
        for (int i = 0; i < kWaves; ++i) there += s.wave[0][i];
        __syncthreads();
        if (there > (u64)top_k) {
            const Cut c = descend<E, false>(row, weights, (u64)top_k, s, wave, lane);
            key = c.key;
            tied = (u64)top_k - c.count;
            cut_ties = tied < c.ties;
            total = c.weight + tied * weights(value_of(key));
        }
    }
    if (top_p < 1) {
        if (key == 0) {
            row.scan(wave * per, (wave + 1) * per < row.groups ? (wave + 1) * per : row.groups, lane,
                     [&](int, float x) { total += weights(x); });
            total = wave_add_u64(total);
            if (lane == 0) s.wave[0][wave] = total;
            __syncthreads();
            total = 0;
            for (int i = 0; i < kWaves; ++i) total += s.wave[0][i];
            __syncthreads();
        }
        const double part = ceil((double)top_p * (double)total);
        const u64 limit = part >= 1 ? (u64)part : 1;
        const Cut c = descend<E, true>(row, weights, limit < total ? limit : total, s, wave, lane);
        const u64 w = weights(value_of(c.key)), need = w ? (limit - c.weight + w - 1) / w : 0;
        const uint32_t before = key;
        key = c.key;
        if (before == key && cut_ties) {
            tied = need < tied ? need : tied;
        } else {
            tied = need < c.ties ? need : c.ties;
            cut_ties = tied < c.ties;
        }
    }
    if (cut_ties) {
        u64 n;
        const uint32_t k = key;
        const u64 want = tied;
        last = locate(row, [&](int, float x) { return (u64)(key_of(x) == k); }, [&](u64) { return want - 1; }, &n, s, wave, lane);
    }
    const auto kept = [&](int id, float x) -> u64 {
        if (x == -INFINITY) return 0;
        const uint32_t k = key_of(x);
        if (k < key || (k == key && id > last)) return 0;
        const u64 w = weights(x);
        return w >= least || id == first ? w : 0;
    };
    const double u = a.u[at];
    const int token = locate(row, kept, [&](u64 all) {
        const double t = u * (double)all;
        return t >= 1 ? (t < (double)all ? (u64)t : all - 1) : 0;
    }, &total, s, wave, lane);
    if (tid == 0) {
        a.tokens[at] = token < 0 ? first : token;
        if (a.logp) {
            const float x = Row<E>::get(((const E*)a.logits)[at * a.V + (token < 0 ? first : token)]);
            a.logp[at] = (float)(((double)x - weights.top) / (double)temperature - log(ldexp((double)total, -shift)));
        }
    }
}

}  // namespace

size_t sample_workspace(int64_t, int, int) { return 0; }

hipError_t launch_sample(const SampleArgs& a, int dtype, void*, hipStream_t stream) {
    int n = 0;
    while ((1ll << n) < a.V) ++n;
    const int shift = 62 - n < 50 ? 62 - n : 50;
    const unsigned rows = (unsigned)((int64_t)a.B * a.rows);
    if (dtype == DT_DTYPE_BF16) sample_kernel<uint16_t><<<rows, kThreads, 0, stream>>>(a, shift);
    else sample_kernel<uint32_t><<<rows, kThreads, 0, stream>>>(a, shift);
    return hipGetLastError();
}

}  // namespace dt
