// Attention over one shared latent vector a token.  The cache holds, for a
// token, a latent c of C elements and a rotated key part r of R elements, the
// same for every query head:
//
//   absorbed (dt_latent_attention)   score = scale (q_c . c + q_r . r),  out = sum p c
//   expanded (dt_latent_prefill)     k = W_k c, v = W_v c for every head,
//                                    score = scale (q_n . k + q_r . r),  out = sum p v
//
// The absorbed form reads C + R elements a key whatever the number of heads and
// spends 2 (2 C + R) operations on a key, row and head; the expanded form
// 2 (2 N + R), after 4 C N a key and head for making k and v.  With C = 512, N =
// 128 and R = 64 that is 2176 against 640 and 262144: the expanded form is the
// cheaper one from about 170 rows on.
//
// The absorbed form has a tile loop of its own (latent_dev.h); the expanded form
// makes its keys and values in the workspace and runs through attention_dev.h's.
// Both share its split of the work and its join.
//
// Measured, expanded (bf16, C = 512, R = 64, N = 128, 32 heads, two chunks of
// 1801-2048 rows over 6-14 K keys, 1.08 T operations): 1245 us, 870 TFLOP/s of
// the 1402 of a large matrix product; make_kernel 298 us of it, attention 940
// (matrix and vector units in turn, as with heads' own keys), the join 25.  A
// chunk of 300 rows over 511 keys and 16 heads 40 us, three dependent launches.
// Keys, values and weights are rounded to the cache's type: the result's error
// against 64 bits is 0.0020-0.0030 in bf16 where fp32 ones leave 0.0017, most of
// which is the result's own rounding.
#include "latent_dev.h"

namespace dt {
namespace {

// ---------------------------------------------------------------------------
// the heads' keys and values from the latents
// ---------------------------------------------------------------------------

constexpr int kMakeTile = 128;     // keys, and rows of the weight, of a workgroup
constexpr int kMakeStep = 64;      // elements of the latents a step
constexpr int kMadeRow = kMakeTile * 2 + 16;   // bytes of a key's results in LDS, spread over the banks

// out[key][n] = sum_i W[n][i] c[key][i] for 128 keys of one request and 128 rows
// of the weight; four waves take 64 x 64 each.  The weight's rows are the left
// operand, so a lane ends with one key and runs of its row.  Bound by the
// way from L2 to LDS and its waits: 298 us for 24 K keys of 32 heads (four buffers
// of 32 elements a step instead of two of 64: the same).
template <class T, int C, int N>
__global__ void __launch_bounds__(256) make_kernel(AttentionArgs a, const uint16_t* weight, uint16_t* made) {
    constexpr int kTile = kMakeTile * kMakeStep * 2, kCopies = kMakeTile / 8 / 4;
    __shared__ __attribute__((aligned(1024))) char lds[4 * kTile];     // two buffers of weights, two of latents
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = blockIdx.z, n0 = blockIdx.y * kMakeTile, k0 = blockIdx.x * kMakeTile;
    static_assert(2 * N % kMakeTile == 0, "a tile of the weight is one head's");
    const Request q = request_of(a, b, 1);
    if (q.rows == 0 || k0 >= q.keys) return;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds);
    const uint16_t* from[kCopies];
    const uint16_t* weights[kCopies];
    const int piece = lane & 7;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int row = (wave * kCopies + i) * 8 + (lane >> 3), at = (piece ^ ((row >> 1) & 7)) * 8;
        const int64_t off = k0 + row < q.keys ? slot_offset(a.kv, b, k0 + row) : -1;
        from[i] = a.kv.k + (off < 0 ? 0 : off) + at;       // a key that is not there is not read later
        weights[i] = weight + (int64_t)(n0 + row) * C + at;
    }
    const auto issue = [&](int s) __attribute__((always_inline)) {
        const uint32_t to = lds0 + (s & 1) * kTile + wave * kCopies * 1024;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            copy_to_lds(weights[i] + s * kMakeStep, to + i * 1024);
            copy_to_lds(from[i] + s * kMakeStep, to + 2 * kTile + i * 1024);
        }
    };
    const int wn = wave & 1, wk = wave >> 1;
    int addr[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) addr[s] = col * 128 + ((2 * s + half) ^ ((col >> 1) & 7)) * 16;
    f32x16 o[2][2] = {};
    issue(0);
    for (int s = 0; s < C / kMakeStep; ++s) {
        wait_copies<0>();
        __syncthreads();
        if (s + 1 < C / kMakeStep) issue(s + 1);
        const char* const wt = lds + (s & 1) * kTile + wn * 64 * 128;
        const char* const xt = lds + 2 * kTile + (s & 1) * kTile + wk * 64 * 128;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            s16x8 w[2], k[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[i] = *(const s16x8*)(wt + addr[x] + i * 32 * 128);
                k[i] = *(const s16x8*)(xt + addr[x] + i * 32 * 128);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) o[i][j] = mfma(T(), w[i], k[j], o[i][j]);
        }
    }
    // through LDS, so that a key's 256 bytes leave together
    static_assert(kMakeTile * kMadeRow <= (int)sizeof(lds), "the results' tile");
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s16x4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = (short)T::put(o[i][j][4 * x + e]);
                *(s16x4*)(lds + (wk * 64 + j * 32 + col) * kMadeRow + (wn * 64 + i * 32 + 8 * x + 4 * half) * 2) = y;
            }
    __syncthreads();
    const int h = n0 / (2 * N);                            // (the tile's rows of the weight are one head's)
    uint16_t* const to = made + ((int64_t)b * a.Hq + h) * a.made_keys * (2 * N) + (n0 - h * 2 * N) + (threadIdx.x & 15) * 8;
#pragma unroll
    for (int i = 0; i < kMakeTile / 16; ++i) {
        const int row = i * 16 + (threadIdx.x >> 4), key = k0 + row;
        if (key < q.keys) *(u32x4*)(to + (int64_t)key * (2 * N)) = *(const u32x4*)(lds + row * kMadeRow + (threadIdx.x & 15) * 16);
    }
}

// ---------------------------------------------------------------------------
// new tokens into the cache
// ---------------------------------------------------------------------------

constexpr int kRotDeep = 4;        // groups of heads of a wave in flight
constexpr int kRotWaves = 2048;    // fewer rows than this are shared by waves

// A wave takes one row, or a part of its heads.  The rotated part of a head is
// R / 8 lanes of 16 bytes; head number Hq is the key's own, which goes to the
// cache.  The first wave of a row also norms the latent, C / 8 lanes.  Bound by
// memory: 7800 rows of 128 heads (249 MB) in 61 us, 4.1 TB/s, of which a copy
// would take 51; one row 9 us, all latency.
template <class T, int C, int R>
__global__ void __launch_bounds__(256) latent_append_kernel(LatentAppendArgs a, int parts) {
    constexpr int kLanes = R / 8, kHeads = 64 / kLanes, kPairs = R / 2;
    __shared__ float2 s_rot[4][kPairs];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t job = (int64_t)blockIdx.x * 4 + wave;
    const int64_t row = job / parts;
    const int part = (int)(job - row * parts);
    if (row >= (int64_t)a.c.B * a.c.rows) return;
    const int b = (int)(row / a.c.rows), r = (int)(row - (int64_t)b * a.c.rows);
    const int l = lane % kLanes, d = l * 8, mine = lane / kLanes, total = a.Hq + 1;

    u32x4 raw[kRotDeep];
    const auto load = [&](int h0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kRotDeep; ++i) {
            const int h = h0 + i * parts * kHeads + mine;
            raw[i] = u32x4{0, 0, 0, 0};
            if (h < total)
                raw[i] = *(const u32x4*)((h < a.Hq ? a.q + row * a.q_stride + h * a.q_head
                                                   : a.rot + row * a.rot_stride) + d);
        }
    };
    const int nn = chunk_nodes(a.c, b);
    if (nn < 0 || r >= a.c.lead + nn) return;
    const int64_t slot = (int64_t)a.c.ctx_len[b] + r;
    load(part * kHeads);
    u32x4 latent = {0, 0, 0, 0};
    if (part == 0 && lane < C / 8) latent = *(const u32x4*)(a.latent + row * a.latent_stride + lane * 8);
    const int64_t at = slot_offset(a.kv, b, slot);
    int64_t pos = slot;
    if (a.c.depths && r >= a.c.lead)
        pos = (int64_t)a.c.ctx_len[b] + a.c.lead - 1 + a.c.depths[(int64_t)b * a.c.n_max + r - a.c.lead];
    if (lane < kPairs) {
        // the angle in fp64, as turns of which only the fraction goes on
        const double turns = a.freqs ? (double)pos * (a.freqs[lane] * 0.15915494309189533577) : 0.0;
        const float t = (float)((turns - rint(turns)) * 2.0);
        float s, c;
        sincospif(t, &s, &c);
        s_rot[wave][lane] = make_float2(c * a.rot_scale, s * a.rot_scale);
    }
    wave_sync();

    if (part == 0 && at >= 0) {
        u32x4 res = latent;
        if (a.norm) {
            float e[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                e[j] = T::get((uint16_t)(latent[j >> 1] >> (16 * (j & 1))));
                sum += e[j] * e[j];
            }
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) sum += __shfl_xor(sum, s);
            const float rs = rsqrtf(sum * (1.0f / C) + a.eps);
            if (lane < C / 8) {
                const u32x4 w = *(const u32x4*)(a.norm + lane * 8);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    res[j] = T::put(e[2 * j] * rs * T::get((uint16_t)w[j])) |
                             (uint32_t)T::put(e[2 * j + 1] * rs * T::get((uint16_t)(w[j] >> 16))) << 16;
            }
        }
        if (lane < C / 8) *(u32x4*)(a.kv.k + at + lane * 8) = res;
    }

    const bool hi = d >= kPairs;
    const int other = (lane + (hi ? -(kLanes / 2) : kLanes / 2)) & 63;
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        cs[j] = s_rot[wave][a.interleaved ? (d + j) >> 1 : (hi ? d - kPairs : d) + j];
        if (!a.interleaved && !hi) cs[j].y = -cs[j].y;     // x cos - other sin, and x cos + other sin
    }
    for (int h0 = part * kHeads; h0 < total; h0 += kRotDeep * parts * kHeads) {
        if (h0 != part * kHeads) load(h0);
#pragma unroll
        for (int i = 0; i < kRotDeep; ++i) {
            const int h = h0 + i * parts * kHeads + mine;
            float e[8], o[8], y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = T::get((uint16_t)(raw[i][j >> 1] >> (16 * (j & 1))));
            if (!a.interleaved) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t p = (uint32_t)__shfl((int)raw[i][j], other);
                    o[2 * j] = T::get((uint16_t)p);
                    o[2 * j + 1] = T::get((uint16_t)(p >> 16));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = e[j] * cs[j].x + o[j] * cs[j].y;
            } else {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    y[j] = e[j] * cs[j].x - e[j + 1] * cs[j].y;
                    y[j + 1] = e[j] * cs[j].y + e[j + 1] * cs[j].x;
                }
            }
            u32x4 res = raw[i];
            if (a.freqs) {
#pragma unroll
                for (int j = 0; j < 4; ++j) res[j] = T::put(y[2 * j]) | (uint32_t)T::put(y[2 * j + 1]) << 16;
            }
            if (h >= total || (h == a.Hq && at < 0)) continue;
            *(u32x4*)((h < a.Hq ? a.q_out + row * a.q_out_stride + h * a.q_out_head : a.kv.v + at) + d) = res;
        }
    }
}

template <class T, int C, int R>
void append_run(const LatentAppendArgs& a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.c.B * a.c.rows;
    const int groups = (a.Hq + 1 + 512 / R - 1) / (512 / R);
    int64_t parts = rows < kRotWaves ? (kRotWaves + rows - 1) / rows : 1;
    if (parts > groups) parts = groups;
    latent_append_kernel<T, C, R><<<(unsigned)((rows * parts + 3) / 4), 256, 0, stream>>>(a, (int)parts);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Calls f with the type and the latent's sizes as constants.
template <class F>
hipError_t with_sizes(int dtype, int C, int R, F f) {
    const auto sizes = [&](auto t) {
        using T = decltype(t);
        if (C == 256) return R == 32 ? f(T(), Latents<256, 32>()) : f(T(), Latents<256, 64>());
        return R == 32 ? f(T(), Latents<512, 32>()) : f(T(), Latents<512, 64>());
    };
    return dtype == DT_DTYPE_BF16 ? sizes(Bf16()) : sizes(F16());
}

// resident workgroups: 64 rows' outputs and queries of C = 512 fill a compute unit
template <int C>
constexpr int kLatentSlots = kCus * (C == 512 ? 1 : 2);

template <class T, int C, int R>
hipError_t run_latent(const AttentionArgs& a, void* workspace, hipStream_t stream) {
    using S = Latent<C, R>;
    const auto kernel = a.by8 ? latent_kernel<T, C, R, true> : latent_kernel<T, C, R, false>;
    return run_kernel<T, C, S::kRows>(kernel, a, 256, S::kLds, kLatentSlots<C>, workspace, stream);
}

int prefill_tile_rows(const ChunkArgs& c) { return c.rows <= 64 ? 64 : 128; }
constexpr int kPrefillSlots = 2 * kCus;

// -1: they pass 63 bits (B and Hq alone stay below 2^31)
int64_t made_bytes(const ChunkArgs& c, int Hq, int N, int keys) {
    int64_t n;
    if (__builtin_mul_overflow((int64_t)c.B * Hq * 2 * N * 2, (int64_t)keys, &n) || n > INT64_MAX - 255) return -1;
    return (n + 255) / 256 * 256;
}

}  // namespace

hipError_t launch_latent_append(const LatentAppendArgs& a, int dtype, int C, int R, hipStream_t stream) {
    return with_sizes(dtype, C, R, [&](auto t, auto l) {
        using L = decltype(l);
        append_run<decltype(t), L::kKey, L::kRot>(a, stream);
        return hipGetLastError();
    });
}

size_t latent_workspace(const ChunkArgs& c, int Hq, int C) {
    const int64_t segments = (int64_t)c.B * (((int64_t)c.rows * Hq + 63) / 64);
    return partial_bytes(segments, C == 512 ? kLatentSlots<512> : kLatentSlots<256>, 64, C);
}

hipError_t launch_latent_attention(const AttentionArgs& a, int dtype, int C, int R, void* workspace, hipStream_t stream) {
    return with_sizes(dtype, C, R, [&](auto t, auto l) {
        using L = decltype(l);
        return run_latent<decltype(t), L::kKey, L::kRot>(a, workspace, stream);
    });
}

size_t prefill_workspace(const ChunkArgs& c, int Hq, int N, int keys) {
    const int mt = prefill_tile_rows(c);
    const int64_t made = made_bytes(c, Hq, N, keys);
    if (made < 0) return SIZE_MAX;
    return (size_t)made +
           partial_bytes((int64_t)c.B * Hq * ((c.rows + mt - 1) / mt), kPrefillSlots, mt, N);
}

hipError_t launch_latent_prefill(AttentionArgs a, const void* weight, int dtype, int C, int R, int N, void* workspace,
                                 hipStream_t stream) {
    return with_sizes(dtype, C, R, [&](auto t, auto l) {
        using T = decltype(t);
        using L = decltype(l);
        uint16_t* const made = (uint16_t*)workspace;
        a.made = made;
        const int keys = a.kv.cap;
        const dim3 grid((unsigned)((keys + kMakeTile - 1) / kMakeTile), (unsigned)((a.Hq * 2 * N + kMakeTile - 1) / kMakeTile),
                        (unsigned)a.c.B);
        if (N == 64) make_kernel<T, L::kKey, 64><<<grid, 256, 0, stream>>>(a, (const uint16_t*)weight, made);
        else make_kernel<T, L::kKey, 128><<<grid, 256, 0, stream>>>(a, (const uint16_t*)weight, made);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        void* const rest = (char*)workspace + made_bytes(a.c, a.Hq, N, a.made_keys);
        const auto go = [&](auto x) {
            using E = decltype(x);
            if (prefill_tile_rows(a.c) == 64) return run<T, E, 2, 2, 1, 32, 2>(a, kPrefillSlots, rest, stream);
            return run<T, E, 4, 1, 1, 64, 2>(a, kPrefillSlots, rest, stream);
        };
        return N == 64 ? go(Expanded<64, L::kRot>()) : go(Expanded<128, L::kRot>());
    });
}

}  // namespace dt
