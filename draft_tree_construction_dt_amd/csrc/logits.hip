// dt_process_logits: penalties for repeated tokens, biases and grammar masks.
//
// A workgroup owns a chunk of the vocabulary for one request and some of its
// rows.  It counts the history's tokens that fall into the chunk in LDS once,
// then streams the chunk of each row through registers, one row ahead.  Counts
// are integers, so the order of the LDS atomics does not matter; of a bias
// listed more than once the largest index wins.  A tree row's path is added to
// the table before its row and taken out behind it, by the few nodes whose
// tokens lie in the chunk at all (most chunks have none).
//
// The kernel is bound by memory: every logit is read and written once.  What
// stands in the way is latency, so the tables are kept small (7 or 8
// workgroups a compute unit): biases are found by their rank among the chunk's
// biased tokens (with a word a token instead the case below took 116 us).
// The counts are kept as [t % 8][t / 8], so that a wave's reads of a vector's
// j-th token are consecutive words whatever the row's alignment.  Measured: 64
// requests x 8 rows of 151936 bf16 logits behind 2048-4096 tokens, half of the
// rows masked, in 92 us (3.5 TB/s; a copy of the same bytes takes 65); the same
// without history, biases and masks 68 us; 64 trees of 64 nodes over the same
// vocabulary 631 us (4.0 TB/s).  Every workgroup scans its request's whole
// history: one row of 151936 logits behind 1000, 10000 and 100000 tokens takes
// 9.7, 14 and 70 us, one row of each of 64 requests 13, 28 and 212.
#include <math.h>

#include "pass.h"
#include "wave.h"

namespace dt {
namespace {

constexpr int kChunk = 4096;               // tokens of a workgroup
constexpr int kWords = kChunk / 32;        // of a bit a token
constexpr int64_t kWorkgroups = 2048;
// A lane goes through its vector's few entries one by one; a wave in which a
// lane has more does all tokens of its vectors at once (16 requests' draft logits
// behind 4096 tokens: chosen 34 us, all at once 39, one by one 39; with 64
// requests memory is the bound and all three take 92).
constexpr int kFew = 3;

template <class T>
struct Io;
template <>
struct Io<float> {
    static constexpr int kVec = 4;
    static __device__ inline float get(const u32x4& v, int j) { return __uint_as_float(v[j]); }
    static __device__ inline void put(u32x4& v, int j, float x) { v[j] = __float_as_uint(x); }
    // ... for a j that is not known when compiled
    static __device__ inline float pick(const u32x4& v, int j) {
        return __uint_as_float(j & 2 ? (j & 1 ? v[3] : v[2]) : (j & 1 ? v[1] : v[0]));
    }
    static __device__ inline void set(u32x4& v, int j, float x) {
#pragma unroll
        for (int w = 0; w < 4; ++w) v[w] = w == j ? __float_as_uint(x) : v[w];
    }
    static __device__ inline float get(float x) { return x; }
    static __device__ inline float put(float x) { return x; }
};
template <>
struct Io<uint16_t> {
    static constexpr int kVec = 8;
    static __device__ inline float get(const u32x4& v, int j) {
        return __uint_as_float(j & 1 ? v[j >> 1] & 0xFFFF0000u : v[j >> 1] << 16);
    }
    static __device__ inline void put(u32x4& v, int j, float x) {
        const uint32_t h = Bf16::put(x);
        v[j >> 1] = j & 1 ? (v[j >> 1] & 0xFFFFu) | h << 16 : (v[j >> 1] & 0xFFFF0000u) | h;
    }
    static __device__ inline uint32_t word(const u32x4& v, int j) {
        return j & 4 ? (j & 2 ? v[3] : v[2]) : (j & 2 ? v[1] : v[0]);
    }
    static __device__ inline float pick(const u32x4& v, int j) {
        return __uint_as_float(j & 1 ? word(v, j) & 0xFFFF0000u : word(v, j) << 16);
    }
    static __device__ inline void set(u32x4& v, int j, float x) {
        const uint32_t h = Bf16::put(x), old = word(v, j), y = j & 1 ? (old & 0xFFFFu) | h << 16 : (old & 0xFFFF0000u) | h;
#pragma unroll
        for (int w = 0; w < 4; ++w) v[w] = w == j >> 1 ? y : v[w];
    }
    static __device__ inline float get(uint16_t x) { return Bf16::get(x); }
    static __device__ inline uint16_t put(float x) { return Bf16::put(x); }
};

// How often each token of the chunk was generated, and a flag (the highest
// bit of its count) for one that occurs in the prompt.
constexpr uint32_t kPrompt = 0x80000000u;
__device__ inline int place(int t) { return (t & 7) * (kChunk / 8) + (t >> 3); }

// Eight bits (of which the caller wants the first few) from bit `at` of a
// bitmap in LDS, `last` the last bit that is wanted.
__device__ inline uint32_t bits_at(const uint32_t* bitmap, int at, int last) {
    const uint8_t* const p = (const uint8_t*)bitmap;
    return (p[at >> 3] | (uint32_t)p[last >> 3] << 8) >> (at & 7);
}

template <class T, bool BIAS>
__global__ void __launch_bounds__(256) logits_kernel(LogitsArgs a) {
    constexpr int kVec = Io<T>::kVec, kPer = kChunk / kVec / 256;    // full vectors of a thread and row
    extern __shared__ uint32_t lds[];
    uint32_t* const s_cnt = lds;
    uint32_t* const s_touched = s_cnt + kChunk;            // tokens with a count, or on some node's path
    uint32_t* const s_biased = s_touched + kWords;         // tokens with a bias
    uint32_t* const s_rank = s_biased + (BIAS ? kWords : 0);         // biased tokens before each 32
    uint32_t* const s_bias = s_rank + (BIAS ? kWords : 0);           // their biases, by rank
    uint32_t* const s_node = s_bias + (BIAS ? (a.n_bias < kChunk ? a.n_bias : kChunk) : 0);  // node << 16 | token
    __shared__ int s_nodes;
    const int b = blockIdx.x, v0 = blockIdx.y * kChunk, tid = threadIdx.x, lane = tid & 63;
    const int len = a.V - v0 < kChunk ? a.V - v0 : kChunk;
    int nn = a.n_nodes ? a.n_nodes[b] : a.n_max;
    nn = nn < 0 ? 0 : (nn > a.n_max ? a.n_max : nn);
    const int rows = a.lead + nn;
    const int step = gridDim.z;
    if ((int)blockIdx.z >= rows) return;

    // A row's vectors begin at its 16-byte boundaries: vector k holds the
    // chunk's tokens k * kVec - miss + 0 .. kVec - 1.  Vectors that reach out
    // of the chunk are done token by token.
    const auto miss_of = [&](int r) { return (int)((((int64_t)b * a.rows + r) * a.V + v0) & (kVec - 1)); };
    // The mask row of this workgroup's i-th row; 64 indexes are read at once, a
    // lane each, so that no row waits for its own.
    int index = -1;
    const auto allow_of = [&](int i) -> const uint8_t* {
        if (!a.allow || (int)blockIdx.z + i * step >= rows) return nullptr;
        const int64_t row0 = (int64_t)b * a.rows + blockIdx.z;
        int64_t at = row0 + (int64_t)i * step;
        if (a.allow_index) {
            const int mine = i + lane;
            if ((i & 63) == 0)
                index = (int)blockIdx.z + mine * step < rows ? a.allow_index[row0 + (int64_t)mine * step] : -1;
            at = __builtin_amdgcn_readlane(index, i & 63);
        }
        return at >= 0 && at < a.allow_rows ? (const uint8_t*)(a.allow + at * ((a.V + 31) >> 5)) : nullptr;
    };
    struct Row {
        u32x4 x[kPer];
        uint8_t lo[kPer], hi[kPer];                        // the mask bytes of a vector's first and last token
    };
    const auto load = [&](int r, const uint8_t* allow, Row& row) {
        const int miss = miss_of(r);
        const T* const in = (const T*)a.logits + ((int64_t)b * a.rows + r) * a.V + v0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int lo = (tid + 256 * u) * kVec - miss;
            if (lo < 0 || lo + kVec > len) continue;
            row.x[u] = *(const u32x4*)(in + lo);
            if (allow) {
                row.lo[u] = allow[(v0 + lo) >> 3];
                row.hi[u] = miss ? allow[(v0 + lo + kVec - 1) >> 3] : 0;
            }
        }
    };
    Row cur;
    int r = blockIdx.z;
    const uint8_t* allow = allow_of(0);
    load(r, allow, cur);

    // the tables
    const int cleared = (int)(s_node - lds);
    for (int i = tid; i < cleared; i += 256) lds[i] = 0;
    if (tid == 0) s_nodes = 0;
    __syncthreads();
    const auto touch = [&](uint32_t t) { atomicOr(&s_touched[t >> 5], 1u << (t & 31)); };
    if (a.history) {
        int n = a.history_len[b];
        n = n < 0 ? 0 : (n > a.history_max ? a.history_max : n);
        const int np = a.prompt_len ? a.prompt_len[b] : 0;
        const int32_t* const h = a.history + (int64_t)b * a.history_max;
        constexpr int kDeep = 8;                           // ids of a thread in flight
        for (int i0 = tid; i0 < n; i0 += kDeep * 256) {
            uint32_t t[kDeep];
#pragma unroll
            for (int j = 0; j < kDeep; ++j) t[j] = i0 + 256 * j < n ? (uint32_t)h[i0 + 256 * j] - (uint32_t)v0 : ~0u;
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                if (t[j] >= (uint32_t)len) continue;
                if (i0 + 256 * j < np) atomicOr(&s_cnt[place((int)t[j])], kPrompt);
                else atomicAdd(&s_cnt[place((int)t[j])], 1u);
                touch(t[j]);
            }
        }
    }
    const int32_t* const bias_ids = a.bias_ids + (int64_t)b * a.n_bias;
    if (BIAS) {
        for (int i = tid; i < a.n_bias; i += 256) {
            const uint32_t t = (uint32_t)bias_ids[i] - (uint32_t)v0;
            if (t < (uint32_t)len) atomicOr(&s_biased[t >> 5], 1u << (t & 31));
        }
    }
    if (a.node_tokens) {
        for (int i = tid; i < nn; i += 256) {
            const uint32_t t = (uint32_t)a.node_tokens[(int64_t)b * a.n_max + i] - (uint32_t)v0;
            if (t >= (uint32_t)len) continue;
            s_node[atomicAdd(&s_nodes, 1)] = (uint32_t)i << 16 | t;
            touch(t);
        }
    }
    __syncthreads();
    const int nodes = s_nodes;
    const auto rank_of = [&](int t) {                      // biased tokens before t
        return (int)s_rank[t >> 5] + __popc(s_biased[t >> 5] & ((1u << (t & 31)) - 1));
    };
    if (BIAS) {
        if (tid < 64) {                                    // two words a lane
            static_assert(kWords == 128, "two words a lane");
            const int x = __popc(s_biased[2 * lane]), y = __popc(s_biased[2 * lane + 1]);
            const int upto = wave_prefix_i32(x + y, lane);
            s_rank[2 * lane] = upto - x - y;
            s_rank[2 * lane + 1] = upto - y;
        }
        __syncthreads();
        for (int i = tid; i < a.n_bias; i += 256) {
            const uint32_t t = (uint32_t)bias_ids[i] - (uint32_t)v0;
            if (t < (uint32_t)len) atomicMax(&s_bias[rank_of((int)t)], (uint32_t)i + 1);
        }
        __syncthreads();
        for (int i = tid; i < (int)(s_node - s_bias); i += 256)      // from the last entry's number to its value
            if (s_bias[i]) s_bias[i] = __float_as_uint(a.bias[(int64_t)b * a.n_bias + s_bias[i] - 1]);
        __syncthreads();
    }
    const float rep = a.repetition ? a.repetition[b] : 1.0f, freq = a.frequency ? a.frequency[b] : 0.0f,
                pres = a.presence ? a.presence[b] : 0.0f;
    // the penalties of token t; false where there are none
    const auto penalise = [&](int t, float& x) {
        const uint32_t c = s_cnt[place(t)], n = c & ~kPrompt;
        const float y = c ? (x > 0 ? x / rep : x * rep) : x;
        x = n ? y - __builtin_fmaf(freq, (float)n, pres) : y;
        return c != 0;
    };

    for (int i = 1; r < rows; r += step, ++i) {
        Row next;
        const uint8_t* const allow_next = allow_of(i);
        if (r + step < rows) load(r + step, allow_next, next);
        const bool path = nodes > 0 && r >= a.lead;
        const auto walk = [&](uint32_t by) {
            const uint32_t* const m = a.node_mask + ((int64_t)b * a.n_max + r - a.lead) * a.mask_words;
            for (int k = tid; k < nodes; k += 256) {
                const uint32_t e = s_node[k], node = e >> 16;
                if (m[node >> 5] >> (node & 31) & 1) atomicAdd(&s_cnt[place((int)(e & 0xFFFF))], by);
            }
        };
        if (path) {
            // The row before, if it has no path, has no barrier of its own: its
            // counts have to be read by every wave before this row's are added.
            if (i > 1 && r - step < a.lead) __syncthreads();
            walk(1u);
            __syncthreads();
        }
        const int miss = miss_of(r);
        const T* const in = (const T*)a.logits + ((int64_t)b * a.rows + r) * a.V + v0;
        T* const out = (T*)a.out + ((int64_t)b * a.rows + r) * a.V + v0;
        const auto single = [&](int t) {
            T y = in[t];
            float x = Io<T>::get(y);
            bool changed = penalise(t, x);
            if (BIAS && s_biased[t >> 5] >> (t & 31) & 1) {
                x += __uint_as_float(s_bias[rank_of(t)]);
                changed = true;
            }
            if (changed) y = Io<T>::put(x);
            if (allow && !(allow[(v0 + t) >> 3] >> ((v0 + t) & 7) & 1)) y = Io<T>::put(-INFINITY);
            out[t] = y;
        };
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int lo = (tid + 256 * u) * kVec - miss;
            if (lo < 0 || lo + kVec > len) {
                for (int t = lo < 0 ? 0 : lo; t < lo + kVec && t < len; ++t) single(t);
                continue;
            }
            u32x4 y = cur.x[u];
            constexpr uint32_t kAll = (1u << kVec) - 1;
            const uint32_t counted = bits_at(s_touched, lo, lo + kVec - 1) & kAll;
            const uint32_t biased = BIAS ? bits_at(s_biased, lo, lo + kVec - 1) & kAll : 0;
            uint32_t todo = counted | biased;
            if (__any(__popc(todo) > kFew)) {
                int rank = 0;
                if (BIAS && biased) rank = rank_of(lo);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    float x = Io<T>::get(cur.x[u], j);
                    bool changed = penalise(lo + j, x);
                    if (BIAS && biased >> j & 1) {
                        x += __uint_as_float(s_bias[rank++]);
                        changed = true;
                    }
                    if (changed) Io<T>::put(y, j, x);
                }
            } else {
                while (todo) {
                    const int j = __builtin_ctz(todo);
                    todo &= todo - 1;
                    float x = Io<T>::pick(y, j);
                    bool changed = penalise(lo + j, x);
                    if (BIAS && biased >> j & 1) {
                        x += __uint_as_float(s_bias[rank_of(lo + j)]);
                        changed = true;
                    }
                    if (changed) Io<T>::set(y, j, x);
                }
            }
            if (allow) {
                const uint32_t ok = (cur.lo[u] | (uint32_t)cur.hi[u] << 8) >> ((v0 + lo) & 7);
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (!(ok >> j & 1)) Io<T>::put(y, j, -INFINITY);
            }
            *(u32x4*)(out + lo) = y;
        }
        if (miss > 0 && tid < miss && kChunk - miss + tid < len) single(kChunk - miss + tid);
        if (path) {
            __syncthreads();
            walk(~0u);
            __syncthreads();
        }
        cur = next;
        allow = allow_next;
    }
}

template <class T>
hipError_t run(const LogitsArgs& a, hipStream_t stream) {
    const int64_t chunks = (a.V + kChunk - 1) / kChunk;
    // a table serves several rows once there are some workgroups a compute unit
    int64_t z = (kWorkgroups + chunks * a.B - 1) / (chunks * a.B);
    z = z < a.rows ? z : a.rows;
    // the chunks of low ids first: they hold most entries and take longest
    // (the draft logits of 64 requests 101 -> 92 us; 32 trees behind 8000 tokens
    // lose: 154 -> 161)
    const dim3 grid((unsigned)a.B, (unsigned)chunks, (unsigned)z);
    const int biases = a.n_bias < kChunk ? a.n_bias : kChunk;
    const size_t words = kChunk + kWords + (a.n_bias > 0 ? 2 * kWords + biases : 0) +
                         (a.node_tokens ? a.n_max : 0);
    if (a.n_bias > 0) logits_kernel<T, true><<<grid, 256, words * 4, stream>>>(a);
    else logits_kernel<T, false><<<grid, 256, words * 4, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, int dtype, hipStream_t stream) {
    return dtype == DT_DTYPE_F32 ? run<float>(a, stream) : run<uint16_t>(a, stream);
}

}  // namespace dt
