// dt_process_logits: penalties for repeated tokens, biases and grammar masks.
//
// A workgroup owns a chunk of the vocabulary for one request: it counts the
// history's tokens that fall into the chunk in LDS once, adds and removes each
// tree row's path, and applies the table to the chunk of every row.  Counts
// are integers, so the order of the LDS atomics does not matter; of a bias
// listed more than once the largest index wins.
#include <math.h>

#include "pass.h"

namespace dt {
namespace {

constexpr int kChunk = 4096;
constexpr uint32_t kPrompt = 0x80000000u;

template <class T>
struct Io;
template <>
struct Io<float> {
    static __device__ inline float get(float x) { return x; }
    static __device__ inline float put(float x) { return x; }
};
template <>
struct Io<uint16_t> {
    static __device__ inline float get(uint16_t x) { return Bf16::get(x); }
    static __device__ inline uint16_t put(float x) { return Bf16::put(x); }
};

template <class T>
__global__ void __launch_bounds__(256) logits_kernel(LogitsArgs a) {
    __shared__ uint32_t s_cnt[kChunk], s_bias[kChunk];
    const int b = blockIdx.y, v0 = blockIdx.x * kChunk, tid = threadIdx.x;
    const int len = a.V - v0 < kChunk ? a.V - v0 : kChunk;
    int nn = a.n_nodes ? a.n_nodes[b] : a.n_max;
    nn = nn < 0 ? 0 : (nn > a.n_max ? a.n_max : nn);
    const int rows = a.lead + nn;
    const int r0 = blockIdx.z;
    if (r0 >= rows) return;
    for (int i = tid; i < kChunk; i += 256) {
        s_cnt[i] = 0;
        s_bias[i] = 0;
    }
    __syncthreads();
    if (a.history) {
        int n = a.history_len[b];
        n = n < 0 ? 0 : (n > a.history_max ? a.history_max : n);
        const int np = a.prompt_len ? a.prompt_len[b] : 0;
        for (int i = tid; i < n; i += 256) {
            const uint32_t t = (uint32_t)(a.history[(int64_t)b * a.history_max + i] - v0);
            if (t >= (uint32_t)len) continue;
            if (i < np) atomicOr(&s_cnt[t], kPrompt);
            else atomicAdd(&s_cnt[t], 1u);
        }
    }
    for (int i = tid; i < a.n_bias; i += 256) {
        const uint32_t t = (uint32_t)(a.bias_ids[(int64_t)b * a.n_bias + i] - v0);
        if (t < (uint32_t)len) atomicMax(&s_bias[t], (uint32_t)i + 1);
    }
    __syncthreads();
    const float rep = a.repetition ? a.repetition[b] : 1.0f, freq = a.frequency ? a.frequency[b] : 0.0f,
                pres = a.presence ? a.presence[b] : 0.0f;
    const int words = (a.V + 31) >> 5;
    for (int r = r0; r < rows; r += gridDim.z) {
        const int64_t row = (int64_t)b * a.rows + r;
        const bool path = a.node_tokens && r >= a.lead;
        const auto walk = [&](uint32_t by) {
            const uint32_t* m = a.node_mask + ((int64_t)b * a.n_max + r - a.lead) * a.mask_words;
            for (int i = tid; i < nn; i += 256) {
                if (!(m[i >> 5] >> (i & 31) & 1)) continue;
                const uint32_t t = (uint32_t)(a.node_tokens[(int64_t)b * a.n_max + i] - v0);
                if (t < (uint32_t)len) atomicAdd(&s_cnt[t], by);
            }
        };
        if (path) {
            walk(1u);
            __syncthreads();
        }
        const uint32_t* allow = nullptr;
        if (a.allow) {
            const int64_t i = a.allow_index ? a.allow_index[row] : row;
            if (i >= 0 && i < a.allow_rows) allow = a.allow + i * words;
        }
        const T* in = (const T*)a.logits + row * a.V + v0;
        T* out = (T*)a.out + row * a.V + v0;
        for (int i = tid; i < len; i += 256) {
            const uint32_t c = s_cnt[i], bi = s_bias[i];
            T y = in[i];
            if (c | bi) {
                float x = Io<T>::get(y);
                const uint32_t n = c & ~kPrompt;
                if (c) x = x > 0 ? x / rep : x * rep;
                if (n) x -= freq * (float)n + pres;
                if (bi) x += a.bias[(int64_t)b * a.n_bias + bi - 1];
                y = Io<T>::put(x);
            }
            if (allow && !(allow[(v0 + i) >> 5] >> ((v0 + i) & 31) & 1)) y = Io<T>::put(-INFINITY);
            out[i] = y;
        }
        if (path) {
            __syncthreads();
            walk(~0u);
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, int dtype, hipStream_t stream) {
    const dim3 grid((a.V + kChunk - 1) / kChunk, a.B, a.rows < 8 ? a.rows : 8);
    if (dtype == DT_DTYPE_F32) logits_kernel<float><<<grid, 256, 0, stream>>>(a);
    else logits_kernel<uint16_t><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace dt
