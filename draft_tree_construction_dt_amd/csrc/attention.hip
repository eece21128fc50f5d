// dt_tree_attention: softmax(scale * q k^T) v over a paged cache, one pass
// over the keys with a running maximum m and sum l:
//   m' = max(m, x);  l' = l e^(m - m') + e^(x - m');  o' = o e^(m - m') + e^(x - m') v
#include <math.h>

#include "pass.h"

namespace dt {
namespace {

// One wave per row and query head; a lane holds D / 64 elements of it.
template <class T, int D>
__global__ void __launch_bounds__(64) attention_simple(AttentionArgs a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x;
    const int h = blockIdx.x % a.Hq;
    const int64_t row = blockIdx.x / a.Hq;
    const int b = (int)(row / a.c.rows), r = (int)(row - (int64_t)b * a.c.rows);
    const int nn = chunk_nodes(a.c, b);
    if (nn < 0 || r >= a.c.lead + nn) return;
    const int64_t ctx = a.c.ctx_len[b];
    const bool node = a.c.mask && r >= a.c.lead;
    const uint32_t* mask = node ? a.c.mask + ((int64_t)b * a.c.n_max + r - a.c.lead) * a.c.mask_words : nullptr;
    int64_t keys = ctx + (node ? a.c.lead + nn : r + 1);
    keys = keys < a.kv.cap ? keys : a.kv.cap;
    float q[E], o[E] = {}, m = -INFINITY, l = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = T::get(a.q[row * a.q_stride + (int64_t)h * D + lane + 64 * e]);
    for (int64_t j = 0; j < keys; ++j) {
        const int64_t i = j - ctx - a.c.lead;
        if (node && i >= 0 && !(mask[i >> 5] >> (i & 31) & 1)) continue;
        const int64_t at = slot_offset(a.kv, b, j);
        if (at < 0) continue;
        const uint16_t* k = a.kv.k + at + (h / a.G) * a.kv.head_stride;
        const uint16_t* v = a.kv.v + at + (h / a.G) * a.kv.head_stride;
        float x = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) x += q[e] * T::get(k[lane + 64 * e]);
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s);
        x *= a.scale_log2;
        const float top = fmaxf(m, x);
        const float base = top == -INFINITY ? 0.0f : top;
        const float w = exp2f(m - base), p = exp2f(x - base);
        m = top;
        l = l * w + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * w + p * T::get(v[lane + 64 * e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        a.out[row * a.out_stride + (int64_t)h * D + lane + 64 * e] = T::put(l == 0 ? 0.0f : o[e] / l);
    if (a.lse && lane == 0) a.lse[row * a.Hq + h] = l == 0 ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <class T>
hipError_t launch_for(const AttentionArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)((int64_t)a.c.B * a.c.rows * a.Hq);
    switch (a.kv.D) {
    case 64: attention_simple<T, 64><<<grid, 64, 0, stream>>>(a); break;
    case 128: attention_simple<T, 128><<<grid, 64, 0, stream>>>(a); break;
    default: attention_simple<T, 256><<<grid, 64, 0, stream>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace

size_t attention_workspace(const ChunkArgs&, int, int, int) { return 256; }

hipError_t launch_attention(const AttentionArgs& a, int dtype, void*, hipStream_t stream) {
    return dtype == DT_DTYPE_BF16 ? launch_for<Bf16>(a, stream) : launch_for<F16>(a, stream);
}

}  // namespace dt
