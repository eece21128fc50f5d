// dt_kv_append: per-head norms of queries and keys, the position rotation, and
// keys and values into their cache slots, in one pass over the projection.
//
// A head is D/8 lanes of 16 bytes, so a wave takes 64 / (D/8) heads at a
// time, kDeep such groups in flight; a wave belongs to one row.  Its angles
// are made once: lane i turns pair i, position * f_i in fp64 (a position times
// a frequency needs more bits than fp32 has from a few thousand positions
// on), as turns, of which only the fraction goes on to an fp32 sine and
// cosine.  The other element of a pair in the half layout lies in a lane
// rot_dim / 16 away: lanes exchange the raw pieces before the norm, two
// elements a word.  Bound by memory (few rows: by latency, so a row is then
// shared by several waves).  Measured: 64 trees of 40-64 nodes, 82.6 MB, in 27 us
// (a copy of the same bytes: 17); 109 MB of prompt in 25 us (4.3 TB/s); one token
// 5.4 us.
#include <math.h>

#include "pass.h"

namespace dt {
namespace {

constexpr int kMaxPairs = 128;     // rot_dim <= 256
constexpr int kDeep = 4;           // groups of heads of a wave in flight
// Fewer rows than this are shared by waves, as many as make about this number.
// Captured calls of 32 + 16 heads of 128, a wave a row / shared: one row 11.2 /
// 5.3 us, 512 rows 14.1 / 8.0, 960 15.6 / 11.5, 1984 18.5 / 17.0.  Up to 8192
// waves instead: 512 rows 11.5, 1984 18.9, 2112 19.3 (a wave a row 20.6), 4160
// the same.
constexpr int kWaves = 2048;

template <class T, int D>
__global__ void __launch_bounds__(256) append_kernel(AppendArgs a, int parts) {
    constexpr int kLanes = D / 8, kHeads = 64 / kLanes;
    __shared__ float2 s_rot[4][kMaxPairs];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t job = (int64_t)blockIdx.x * 4 + wave;
    const int64_t row = job / parts;
    const int part = (int)(job - row * parts);
    if (row >= (int64_t)a.c.B * a.c.rows) return;
    const int b = (int)(row / a.c.rows), r = (int)(row - (int64_t)b * a.c.rows);
    const int nq = a.Hq, nk = nq + a.kv.Hkv, total = nk + a.kv.Hkv;
    const int l = lane % kLanes, d = l * 8, mine = lane / kLanes;
    const int half = a.rot_dim >> 1;

    // A group of heads, 16 bytes a lane.
    struct Head {
        u32x4 raw;
        int h;
    };
    const auto load = [&](int h0, Head (&x)[kDeep]) {
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int h = h0 + i * parts * kHeads + mine;
            const uint16_t* src = h < nq ? a.q + row * a.q_stride + (int64_t)h * D
                                         : (h < nk ? a.k + row * a.k_stride + (int64_t)(h - nq) * D
                                                   : a.v + row * a.v_stride + (int64_t)(h - nk) * D);
            x[i].h = h;
            x[i].raw = u32x4{0, 0, 0, 0};
            if (h < total) x[i].raw = *(const u32x4*)(src + d);
        }
    };
    const int nn = chunk_nodes(a.c, b);
    if (nn < 0 || r >= a.c.lead + nn) return;
    const int64_t slot = (int64_t)a.c.ctx_len[b] + r;
    Head x[kDeep];
    load(part * kHeads, x);
    const int64_t at = slot_offset(a.kv, b, slot);
    int64_t pos = slot;
    if (a.c.depths && r >= a.c.lead)
        pos = (int64_t)a.c.ctx_len[b] + a.c.lead - 1 + a.c.depths[(int64_t)b * a.c.n_max + r - a.c.lead];
    for (int i = lane; i < half; i += 64) {
        const double turns = (double)pos * (a.freqs[i] * 0.15915494309189533577);
        const float t = (float)((turns - rint(turns)) * 2.0);
        float s, c;
        sincospif(t, &s, &c);
        s_rot[wave][i] = make_float2(c * a.rot_scale, s * a.rot_scale);
    }
    wave_sync();
    // this lane's angles and norm weights, the same for every head
    const bool turn = d < a.rot_dim, hi = d >= half;
    const int other = (lane + (hi ? -(half >> 3) : half >> 3)) & 63, od = hi ? d - half : d + half;
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = a.interleaved ? (d + j) >> 1 : (hi ? d - half : d) + j;
        cs[j] = turn ? s_rot[wave][i & (kMaxPairs - 1)] : make_float2(1, 0);
        if (turn && !a.interleaved && !hi) cs[j].y = -cs[j].y;         // x cos - other sin, and x cos + other sin
    }
    for (int h0 = part * kHeads; h0 < total; h0 += kDeep * parts * kHeads) {
        if (h0 != part * kHeads) load(h0, x);
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int h = x[i].h;
            const bool is_q = h < nq, is_k = !is_q && h < nk;
            const uint16_t* w = is_q ? a.q_norm : (is_k ? a.k_norm : nullptr);
            const u32x4 raw = x[i].raw;
            float e[8], o[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                e[j] = T::get((uint16_t)(raw[j >> 1] >> (16 * (j & 1))));
                sum += e[j] * e[j];
            }
#pragma unroll
            for (int s = 1; s < kLanes; s <<= 1) sum += __shfl_xor(sum, s);
            if (!a.interleaved) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t p = (uint32_t)__shfl((int)raw[j], other);
                    o[2 * j] = T::get((uint16_t)p);
                    o[2 * j + 1] = T::get((uint16_t)(p >> 16));
                }
            }
            if (w) {
                const float rs = rsqrtf(sum * (1.0f / D) + a.eps);
                const u32x4 we = *(const u32x4*)(w + d);
                u32x4 wo = we;
                if (!a.interleaved && turn) wo = *(const u32x4*)(w + od);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    e[j] = e[j] * rs * T::get((uint16_t)(we[j >> 1] >> (16 * (j & 1))));
                    if (!a.interleaved) o[j] = o[j] * rs * T::get((uint16_t)(wo[j >> 1] >> (16 * (j & 1))));
                }
            }
            u32x4 res = raw;
            if ((is_q || is_k) && (w || turn)) {
                float y[8];
                if (!a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = turn ? e[j] * cs[j].x + o[j] * cs[j].y : e[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        y[j] = turn ? e[j] * cs[j].x - e[j + 1] * cs[j].y : e[j];
                        y[j + 1] = turn ? e[j] * cs[j].y + e[j + 1] * cs[j].x : e[j + 1];
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) res[j] = T::put(y[2 * j]) | (uint32_t)T::put(y[2 * j + 1]) << 16;
            }
            if (h >= total || (!is_q && at < 0)) continue;
            uint16_t* dst = is_q ? a.q_out + row * a.q_out_stride + (int64_t)h * D
                                 : (is_k ? a.kv.k : a.kv.v) + at + (is_k ? h - nq : h - nk) * a.kv.head_stride;
            *(u32x4*)(dst + d) = res;
        }
    }
}

template <class T, int D>
void run(const AppendArgs& a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.c.B * a.c.rows;
    const int groups = (a.Hq + 2 * a.kv.Hkv + 512 / D - 1) / (512 / D);      // of 64 / (D / 8) heads
    int64_t parts = rows < kWaves ? (kWaves + rows - 1) / rows : 1;
    if (parts > groups) parts = groups;
    append_kernel<T, D><<<(unsigned)((rows * parts + 3) / 4), 256, 0, stream>>>(a, (int)parts);
}

template <class T>
hipError_t launch_for(const AppendArgs& a, hipStream_t stream) {
    switch (a.kv.D) {
    case 64: run<T, 64>(a, stream); break;
    case 128: run<T, 128>(a, stream); break;
    default: run<T, 256>(a, stream); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, int dtype, hipStream_t stream) {
    return dtype == DT_DTYPE_BF16 ? launch_for<Bf16>(a, stream) : launch_for<F16>(a, stream);
}

}  // namespace dt
