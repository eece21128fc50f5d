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
// The kernel is bound by memory: every logit is read and written once, and the
// table costs its LDS reads (8 words of 16 bytes read).  The table is kept as
// [t % 8][t / 8], so that a wave's reads of a vector's j-th token are
// consecutive words whatever the row's alignment.
#include <math.h>

#include "pass.h"

namespace dt {
namespace {

constexpr uint32_t kPrompt = 0x80000000u;  // the token occurs in the prompt
constexpr int kMaxNodes = kMaxCommitNodes;
constexpr int64_t kWorkgroups = 2048;

template <class T>
struct Io;
template <>
struct Io<float> {
    static constexpr int kVec = 4;
    static __device__ inline float get(const u32x4& v, int j) { return __uint_as_float(v[j]); }
    static __device__ inline void put(u32x4& v, int j, float x) { v[j] = __float_as_uint(x); }
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
    static __device__ inline float get(uint16_t x) { return Bf16::get(x); }
    static __device__ inline uint16_t put(float x) { return Bf16::put(x); }
};

template <class T, int CHUNK, bool BIAS>
__global__ void __launch_bounds__(256) logits_kernel(LogitsArgs a) {
    constexpr int kVec = Io<T>::kVec, kPer = CHUNK / kVec / 256;     // full vectors of a thread and row
    __shared__ uint32_t s_cnt[CHUNK];
    __shared__ uint32_t s_bias[BIAS ? CHUNK : 1];
    __shared__ uint32_t s_node[kMaxNodes];                 // node << 16 | place in the chunk
    __shared__ int s_nodes;
    const int b = blockIdx.y, v0 = blockIdx.x * CHUNK, tid = threadIdx.x;
    const int len = a.V - v0 < CHUNK ? a.V - v0 : CHUNK;
    int nn = a.n_nodes ? a.n_nodes[b] : a.n_max;
    nn = nn < 0 ? 0 : (nn > a.n_max ? a.n_max : nn);
    const int rows = a.lead + nn;
    const int step = gridDim.z;
    if ((int)blockIdx.z >= rows) return;
    const auto place = [](int t) { return (t & 7) * (CHUNK / 8) + (t >> 3); };

    // A row's vectors begin at its 16-byte boundaries: vector k holds the
    // chunk's tokens k * kVec - miss + 0 .. kVec - 1.  Vectors that reach out
    // of the chunk are done token by token.
    const auto miss_of = [&](int r) { return (int)((((int64_t)b * a.rows + r) * a.V + v0) & (kVec - 1)); };
    const auto allow_of = [&](int r) -> const uint8_t* {
        if (!a.allow || r >= rows) return nullptr;
        const int64_t row = (int64_t)b * a.rows + r;
        const int64_t i = a.allow_index ? a.allow_index[row] : row;
        return i >= 0 && i < a.allow_rows ? (const uint8_t*)(a.allow + i * ((a.V + 31) >> 5)) : nullptr;
    };
    struct Row {
        u32x4 x[kPer];
        uint32_t ok[kPer];
    };
    const auto load = [&](int r, const uint8_t* allow, Row& row) {
        const int miss = miss_of(r);
        const T* const in = (const T*)a.logits + ((int64_t)b * a.rows + r) * a.V + v0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int lo = (tid + 256 * u) * kVec - miss;
            row.ok[u] = ~0u;
            if (lo < 0 || lo + kVec > len) continue;
            row.x[u] = *(const u32x4*)(in + lo);
            if (allow) {
                const int bit = v0 + lo, last = (bit + kVec - 1) >> 3;
                row.ok[u] = (allow[bit >> 3] | (uint32_t)allow[last] << 8) >> (bit & 7);
                if (last == bit >> 3) row.ok[u] = (uint32_t)allow[last] >> (bit & 7);
            }
        }
    };
    Row cur;
    int r = blockIdx.z;
    const uint8_t* allow = allow_of(r);
    load(r, allow, cur);

    for (int i = tid; i < CHUNK; i += 256) {
        s_cnt[i] = 0;
        if (BIAS) s_bias[i] = 0;
    }
    if (tid == 0) s_nodes = 0;
    __syncthreads();
    if (a.history) {
        int n = a.history_len[b];
        n = n < 0 ? 0 : (n > a.history_max ? a.history_max : n);
        const int np = a.prompt_len ? a.prompt_len[b] : 0;
        const int32_t* const h = a.history + (int64_t)b * a.history_max;
        for (int i0 = tid; i0 < n; i0 += 4 * 256) {
            uint32_t t[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = i0 + 256 * j < n ? (uint32_t)(h[i0 + 256 * j] - v0) : ~0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (t[j] >= (uint32_t)len) continue;
                uint32_t* const c = &s_cnt[place((int)t[j])];
                if (i0 + 256 * j < np) atomicOr(c, kPrompt);
                else atomicAdd(c, 1u);
            }
        }
    }
    if (BIAS) {
        for (int i = tid; i < a.n_bias; i += 256) {
            const uint32_t t = (uint32_t)(a.bias_ids[(int64_t)b * a.n_bias + i] - v0);
            if (t < (uint32_t)len) atomicMax(&s_bias[place((int)t)], (uint32_t)i + 1);
        }
    }
    if (a.node_tokens) {
        for (int i = tid; i < nn; i += 256) {
            const uint32_t t = (uint32_t)(a.node_tokens[(int64_t)b * a.n_max + i] - v0);
            if (t < (uint32_t)len) s_node[atomicAdd(&s_nodes, 1)] = (uint32_t)i << 16 | t;
        }
    }
    __syncthreads();
    const int nodes = s_nodes;
    const float rep = a.repetition ? a.repetition[b] : 1.0f, freq = a.frequency ? a.frequency[b] : 0.0f,
                pres = a.presence ? a.presence[b] : 0.0f, inv = 1.0f / rep;
    // token t of the chunk; false where nothing touches it
    const auto apply = [&](int t, float& x) {
        const uint32_t c = s_cnt[place(t)], bi = BIAS ? s_bias[place(t)] : 0;
        const float n = (float)(c & ~kPrompt);
        const float y = c ? x * (x > 0 ? inv : rep) : x;
        x = (c & ~kPrompt) ? y - __builtin_fmaf(freq, n, pres) : y;
        if (BIAS && bi) x += a.bias[(int64_t)b * a.n_bias + bi - 1];
        return (c | bi) != 0;
    };

    for (; r < rows; r += step) {
        Row next;
        const uint8_t* const allow_next = allow_of(r + step);
        if (r + step < rows) load(r + step, allow_next, next);
        const bool path = nodes > 0 && r >= a.lead;
        const auto walk = [&](uint32_t by) {
            const uint32_t* const m = a.node_mask + ((int64_t)b * a.n_max + r - a.lead) * a.mask_words;
            for (int i = tid; i < nodes; i += 256) {
                const uint32_t e = s_node[i], node = e >> 16;
                if (m[node >> 5] >> (node & 31) & 1) atomicAdd(&s_cnt[place((int)(e & 0xFFFF))], by);
            }
        };
        if (path) {
            walk(1u);
            __syncthreads();
        }
        const int miss = miss_of(r);
        const T* const in = (const T*)a.logits + ((int64_t)b * a.rows + r) * a.V + v0;
        T* const out = (T*)a.out + ((int64_t)b * a.rows + r) * a.V + v0;
        const auto single = [&](int t) {
            T y = in[t];
            float x = Io<T>::get(y);
            if (apply(t, x)) y = Io<T>::put(x);
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
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                float x = Io<T>::get(cur.x[u], j);
                if (apply(lo + j, x)) Io<T>::put(y, j, x);
                if (!(cur.ok[u] >> j & 1)) Io<T>::put(y, j, -INFINITY);
            }
            *(u32x4*)(out + lo) = y;
        }
        if (miss > 0 && tid < miss && CHUNK - miss + tid < len) single(CHUNK - miss + tid);
        if (path) {
            __syncthreads();
            walk(~0u);
            __syncthreads();
        }
        cur = next;
        allow = allow_next;
    }
}

template <class T, int CHUNK>
hipError_t run(const LogitsArgs& a, hipStream_t stream) {
    const int64_t chunks = (a.V + CHUNK - 1) / CHUNK;
    // a table serves several rows once there are some workgroups a compute unit
    int64_t z = (kWorkgroups + chunks * a.B - 1) / (chunks * a.B);
    z = z < a.rows ? z : a.rows;
    const dim3 grid((unsigned)chunks, (unsigned)a.B, (unsigned)z);
    if (a.n_bias > 0) logits_kernel<T, CHUNK, true><<<grid, 256, 0, stream>>>(a);
    else logits_kernel<T, CHUNK, false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, int dtype, hipStream_t stream) {
    if (dtype == DT_DTYPE_F32) return run<float, 4096>(a, stream);
    return run<uint16_t, 4096>(a, stream);
}

}  // namespace dt
