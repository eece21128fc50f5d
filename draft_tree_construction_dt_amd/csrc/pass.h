// The verification pass over a built tree (dt.h, second part): what its
// kernels share on the device, their arguments, and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dt.h"

namespace dt {

// Chunk of new tokens, as dt_chunk; rows = lead + n_max.
struct ChunkArgs {
    int B, lead, n_max, rows, mask_words;
    const int32_t* ctx_len;
    const int32_t* n_nodes;
    const uint32_t* mask;
    const int32_t* depths;
};

// One layer of a paged cache (k and v point at it).
struct CacheArgs {
    uint16_t* k;
    uint16_t* v;
    const int32_t* page_table;
    int64_t page_stride, slot_stride, head_stride;
    int num_pages, page_size, max_pages, Hkv, D;
    int cap;                       // max_pages * page_size
    int page_shift;                // log2(page_size), or -1 where it is no power of two
};

struct AppendArgs {
    ChunkArgs c;
    CacheArgs kv;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int Hq;
    const uint16_t* q_norm;
    const uint16_t* k_norm;
    float eps, rot_scale;
    const double* freqs;
    int rot_dim, interleaved;
};

struct AttentionArgs {
    ChunkArgs c;
    CacheArgs kv;
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride;
    int Hq, G;
    float scale_log2;              // scale * log2(e)
    bool by8;                      // slots 8 n .. 8 n + 7 lie in one page, within 2^31 bytes
    float* lse;
};

struct LogitsArgs {
    const void* logits;
    void* out;
    int B, lead, n_max, rows, V, mask_words;
    const int32_t* n_nodes;
    const int32_t* history;
    int history_max;
    const int32_t* history_len;
    const int32_t* prompt_len;
    const int32_t* node_tokens;
    const uint32_t* node_mask;
    const float* repetition;
    const float* frequency;
    const float* presence;
    const int32_t* bias_ids;
    const float* bias;
    int n_bias;
    const uint32_t* allow;
    const int32_t* allow_index;
    int allow_rows;
};

struct CommitArgs {
    ChunkArgs c;
    CacheArgs kv;                  // k = v = NULL: tokens only
    int64_t layer_stride;
    int layers;
    const int32_t* tokens;
    const int32_t* parents;
    const int32_t* target;
    int L;
    int32_t* accepted;
    int32_t* lengths;
    int32_t* nodes;
};

constexpr int kMaxChunkRows = 65536;
constexpr int64_t kMaxBatchRows = 1 << 24;
constexpr int kMaxPassHeads = 4096;
constexpr int kMaxCommitNodes = 1024;
constexpr int64_t kMaxSlots = 1 << 30;

hipError_t launch_append(const AppendArgs& a, int dtype, hipStream_t stream);
hipError_t launch_attention(const AttentionArgs& a, int dtype, void* workspace, hipStream_t stream);
size_t attention_workspace(const ChunkArgs& c, int Hkv, int Hq, int D);
hipError_t launch_logits(const LogitsArgs& a, int dtype, hipStream_t stream);
hipError_t launch_commit(const CommitArgs& a, hipStream_t stream);

#ifdef __HIPCC__

// Nodes of request b that count, and -1 for a request without rows.
__device__ inline int chunk_nodes(const ChunkArgs& c, int b) {
    if (c.ctx_len[b] < 0) return -1;
    if (!c.n_nodes) return c.n_max;
    const int n = c.n_nodes[b];
    return n < 0 ? 0 : (n > c.n_max ? c.n_max : n);
}

// Element offset of the token in `slot` of request b (head 0), or -1 where
// the cache has no such token.  64 bits: caches pass 2^31 elements.
__device__ inline int64_t slot_offset(const CacheArgs& kv, int b, int64_t slot) {
    if (slot >= kv.cap) return -1;
    const int s = (int)slot;
    const int i = kv.page_shift >= 0 ? s >> kv.page_shift : s / kv.page_size;
    const int page = kv.page_table[(int64_t)b * kv.max_pages + i];
    if (page < 0 || page >= kv.num_pages) return -1;
    return page * kv.page_stride + (s - i * kv.page_size) * kv.slot_stride;
}

// The two 16-bit types of heads.
struct Bf16 {
    static constexpr uint32_t kExponent = 0x7F80, kFraction = 0x007F, kOne = 0x3F80, k256 = 0x4380;
    static __device__ inline float get(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
    static __device__ inline uint16_t put(float x) {
        const __bf16 h = (__bf16)x;                  // to nearest, ties to even
        return __builtin_bit_cast(uint16_t, h);
    }
};
struct F16 {
    static constexpr uint32_t kExponent = 0x7C00, kFraction = 0x03FF, kOne = 0x3C00, k256 = 0x5C00;
    static __device__ inline float get(uint16_t x) { return (float)__builtin_bit_cast(_Float16, x); }
    static __device__ inline uint16_t put(float x) {
        const _Float16 h = (_Float16)x;
        return __builtin_bit_cast(uint16_t, h);
    }
};

// Orders a wave's LDS accesses without a workgroup barrier.
__device__ inline void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#endif

}  // namespace dt
