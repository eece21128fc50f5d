// dt_kv_append: per-head norms of queries and keys, the position rotation, and
// keys and values into their cache slots, in one pass over the projection.
//
// A head is D/8 lanes of 16 bytes, so a wave takes 64 / (D/8) heads at a
// time; a wave belongs to one row.  Its angles are made once: lane i turns
// pair i, position * f_i in fp64 (a position times a frequency needs more
// bits than fp32 has from a few thousand positions on), as turns, of which
// only the fraction goes on to an fp32 sine and cosine.
#include <math.h>

#include "pass.h"

namespace dt {
namespace {

constexpr int kMaxPairs = 128;     // rot_dim <= 256

template <class T, int D>
__global__ void __launch_bounds__(256) append_kernel(AppendArgs a, int parts) {
    constexpr int kLanes = D / 8, kHeads = 64 / kLanes;
    __shared__ float2 s_rot[4][kMaxPairs];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t job = (int64_t)blockIdx.x * 4 + wave;
    const int64_t row = job / parts;
    const int part = (int)(job - row * parts);
    if (row >= (int64_t)a.c.B * a.c.rows) return;
    const int b = (int)(row / a.c.rows), r = (int)(row - (int64_t)b * a.c.rows);
    const int nn = chunk_nodes(a.c, b);
    if (nn < 0 || r >= a.c.lead + nn) return;
    const int64_t slot = (int64_t)a.c.ctx_len[b] + r;
    const int64_t at = slot_offset(a.kv, b, slot);
    int64_t pos = slot;
    if (a.c.depths && r >= a.c.lead)
        pos = (int64_t)a.c.ctx_len[b] + a.c.lead - 1 + a.c.depths[(int64_t)b * a.c.n_max + r - a.c.lead];
    const int half = a.rot_dim >> 1;
    for (int i = lane; i < half; i += 64) {
        const double turns = (double)pos * (a.freqs[i] * 0.15915494309189533577);
        const float x = (float)((turns - rint(turns)) * 2.0);
        float s, c;
        sincospif(x, &s, &c);
        s_rot[wave][i] = make_float2(c * a.rot_scale, s * a.rot_scale);
    }
    wave_sync();
    const int total = (a.q ? a.Hq : 0) + 2 * a.kv.Hkv, nq = a.q ? a.Hq : 0;
    const int l = lane % kLanes, d = l * 8;
    for (int h0 = part * kHeads; h0 < total; h0 += parts * kHeads) {
        const int h = h0 + lane / kLanes;
        const bool is_q = h < nq, is_k = !is_q && h < nq + a.kv.Hkv, live = h < total;
        const int hk = is_q ? 0 : (is_k ? h - nq : h - nq - a.kv.Hkv);
        const uint16_t* src = is_q ? a.q + row * a.q_stride + (int64_t)h * D
                                   : (is_k ? a.k + row * a.k_stride : a.v + row * a.v_stride) + (int64_t)hk * D;
        u32x4 raw = {0, 0, 0, 0};
        if (live) raw = *(const u32x4*)(src + d);
        const uint16_t* w = is_q ? a.q_norm : (is_k ? a.k_norm : nullptr);
        float x[8];
        float sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = T::get((uint16_t)(raw[j >> 1] >> (16 * (j & 1))));
            sum += x[j] * x[j];
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor(sum, o);
        if (w) {
            const float rs = rsqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * rs * T::get(w[d + j]);
        }
        const bool turn = (is_q || is_k) && d < a.rot_dim;
        float y[8];
        if (!a.interleaved) {
            const bool hi = d >= half;
            const int other = lane + (hi ? -(half >> 3) : half >> 3);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = __shfl(x[j], other & 63);
                y[j] = x[j];
                if (turn) {
                    const float2 cs = s_rot[wave][(hi ? d - half : d) + j];
                    y[j] = x[j] * cs.x + (hi ? p * cs.y : -p * cs.y);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                y[j] = x[j];
                y[j + 1] = x[j + 1];
                if (turn) {
                    const float2 cs = s_rot[wave][(d + j) >> 1];
                    y[j] = x[j] * cs.x - x[j + 1] * cs.y;
                    y[j + 1] = x[j] * cs.y + x[j + 1] * cs.x;
                }
            }
        }
        u32x4 res = raw;
        if (is_q || is_k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) res[j] = T::put(y[2 * j]) | (uint32_t)T::put(y[2 * j + 1]) << 16;
        }
        if (!live || (!is_q && at < 0)) continue;
        uint16_t* dst = is_q ? a.q_out + row * a.q_out_stride + (int64_t)h * D
                             : (is_k ? a.kv.k : a.kv.v) + at + hk * a.kv.head_stride;
        *(u32x4*)(dst + d) = res;
    }
}

template <class T>
hipError_t launch_for(const AppendArgs& a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.c.B * a.c.rows;
    const int parts = 1;
    const unsigned grid = (unsigned)((rows * parts + 3) / 4);
    switch (a.kv.D) {
    case 64: append_kernel<T, 64><<<grid, 256, 0, stream>>>(a, parts); break;
    case 128: append_kernel<T, 128><<<grid, 256, 0, stream>>>(a, parts); break;
    default: append_kernel<T, 256><<<grid, 256, 0, stream>>>(a, parts); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, int dtype, hipStream_t stream) {
    return dtype == DT_DTYPE_BF16 ? launch_for<Bf16>(a, stream) : launch_for<F16>(a, stream);
}

}  // namespace dt
