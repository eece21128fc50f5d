// Attention over a paged cache in one pass over the keys: the split of the
// work, the tile loop and the join of partial results, for heads whose keys and
// values are cached (attention.hip) and for latents (latent.hip).
#pragma once

#include <math.h>

#include "pass.h"
#include "wave.h"

namespace dt {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef uint64_t u64;

constexpr int kUnit = 64;          // keys of the split's unit of work
constexpr int kMinUnits = 4;       // a chunk has at least 256 keys
constexpr float kOneRound = 16;    // units a slot up to which the work is cut into one round
constexpr float kSplitCost = 4;    // a partial result's way through memory, in units
// Requests up to which the chunk's size is searched for.  Every workgroup reads
// the batch's lengths and searches for itself, so both grow with the square of
// the batch: one token over 4000 keys (pages of a small pool) for each of 64
// requests 164 us, 256 753, 512 1947, 513 (no search) 1106, 1024 2450; over 100
// keys 64 26, 256 333, 512 1148, 513 340, 4096 11 ms; 65535 of one key 1.4 s.
constexpr int kMaxSearch = 512;
constexpr float kMaxUnits = (float)(kMaxSlots / kUnit);    // no segment has more: sizes stay far from int's end
constexpr int kRowsPerWave = 32;
constexpr float kLazy = 8.0f;      // log2 of how far the maximum may run ahead of the sums

// f16 has no weights below 2^-24 and full ones from 2^-14 only, so its weights
// are 2^kLift times e^(score - maximum): they reach 2^15, just inside the type,
// and a key at 2^-21 of the largest is still as exact as any, one at 2^-31
// still there (262144 keys at 2^-25 beside one of weight 1 lost 1.1% of the
// result without).  bf16's exponents need none.  Scores from kFar on are
// themselves off by so much that weights could pass the type: those are not
// lifted, and the sums follow every larger score.
constexpr float kLift = 7.0f;
constexpr float kFar = 1048576.0f;
__device__ inline float lift(Bf16, float) { return 0.0f; }
__device__ inline float lift(F16, float top) { return fabsf(top) < kFar ? kLift : 0.0f; }
// log2 of the largest weight before the sums are rescaled
__device__ inline float room(Bf16, float) { return kLazy; }
__device__ inline float room(F16, float m) { return fabsf(m) < kFar ? kLazy + kLift : 0.0f; }

__device__ inline f32x16 mfma(Bf16, s16x8 a, s16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b16x8, a), __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
}
__device__ inline f32x16 mfma(F16, s16x8 a, s16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h16x8, a), __builtin_bit_cast(h16x8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// the split
// ---------------------------------------------------------------------------

struct Request {
    int rows, mtiles, units;       // live chunk rows, row tiles, key units
    int keys;
};

__device__ inline Request request_of(const AttentionArgs& a, int b, int mt_rows) {
    Request q{};
    const int nn = b < a.c.B ? chunk_nodes(a.c, b) : -1;
    if (nn < 0) return q;
    q.rows = a.c.lead + nn;
    const int64_t keys = (int64_t)a.c.ctx_len[b] + q.rows;
    q.keys = (int)(keys < a.kv.cap ? keys : a.kv.cap);
    q.mtiles = (q.rows * a.G + mt_rows - 1) / mt_rows;
    q.units = (q.keys + kUnit - 1) / kUnit;
    return q;
}

__device__ inline int64_t uniform(int64_t x) {
    return (int64_t)((u64)(uint32_t)__builtin_amdgcn_readfirstlane((int)x) |
                     (u64)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32);
}

// Units of a chunk: the same on every wave of every workgroup of a call.
// `slots` workgroups are resident at a time, so J chunks of c units take
// about ceil(J / slots) * (c + kSplitCost) units of time.  Work of a few units
// a slot is cut into one round; more into the best of 64 sizes, a lane each,
// around one to four rounds.  `q0`: the first 64 requests.
__device__ inline int chunk_units(const AttentionArgs& a, const Request& q0, int mt_rows, int slots, int lane) {
    double work = 0;
    int segs = 0, longest = 0;
    for (int b0 = 0; b0 < a.c.B; b0 += 64) {
        const Request q = b0 ? request_of(a, b0 + lane, mt_rows) : q0;
        segs += q.mtiles * a.kv.Hkv;
        work += (double)(q.mtiles * a.kv.Hkv) * q.units;
        longest = q.units > longest ? q.units : longest;
    }
    segs = wave_add_i32(segs);
    work = wave_add_f64(work);
    longest = -wave_min_i32(-longest);
    const float each = (float)work / (float)slots;         // units a slot
    if (each < kOneRound || a.c.B > kMaxSearch) {
        // rounding adds at most one chunk a segment
        const int room = 2 * segs < slots ? slots - segs : slots;
        const int c = (int)fminf((float)work / (float)room, kMaxUnits) + 1;
        return c < kMinUnits ? kMinUnits : c;
    }
    // sizes each * (1 .. 1.94) / (1 .. 4); the longest segment whole is one, too
    const float want = fminf(each * (1.0f + 0.0625f * (lane & 15)) / (float)(1 + (lane >> 4)), kMaxUnits);
    int c = lane == 0 ? longest : (int)want + 1;
    c = c < kMinUnits ? kMinUnits : c;
    const float inv = 1.0f / (float)c;
    int jobs = 0;
    for (int b0 = 0; b0 < a.c.B; b0 += 64) {
        const Request q = b0 ? request_of(a, b0 + lane, mt_rows) : q0;
        const int n = a.c.B - b0 < 64 ? a.c.B - b0 : 64;
        for (int i = 0; i < n; ++i) {
            const int u = __builtin_amdgcn_readlane(q.units, i), m = __builtin_amdgcn_readlane(q.mtiles, i);
            jobs += m * a.kv.Hkv * (int)((float)(u + c - 1) * inv);
        }
    }
    const int rounds = (jobs + slots - 1) / slots;
    const int most = longest < c ? longest : c;
    const float cost = (float)rounds * ((float)most + (longest > c ? kSplitCost : 0.0f));
    // the cheapest; of equals the largest size (fewest partial results)
    const float best = wave_min_f32(cost);
    return -wave_min_i32(cost == best ? -c : 0);
}

__device__ inline int splits_of(const Request& q, int c) { return (q.units + c - 1) / c; }

// Partial results of a request: those of its chunks, if its segments are
// split.  A segment of u > c units has fewer than u / c + 1 < 2 u / c chunks, a
// call thus fewer than work / c + (split segments) of them, and fewer split
// segments than work / c; c is more than work / (4 slots).
__device__ inline int partials_of(const AttentionArgs& a, const Request& q, int splits) {
    return splits > 1 ? q.mtiles * a.kv.Hkv * splits : 0;
}

// Row tiles of nearly equal size: the blocks of 32 rows are dealt out so that
// tiles differ by one block at most (trees of 64 nodes and a root with four
// heads to a key head have 260 rows: three tiles of three blocks instead of
// 4, 4 and 1).  The first `more` tiles have base + 1 blocks.
struct Tiling {
    int base, more;
};
__device__ inline Tiling tiling_of(int mrows, int mtiles) {
    const int blocks = (mrows + kRowsPerWave - 1) / kRowsPerWave, base = blocks / mtiles;
    return {base, blocks - base * mtiles};
}

struct Job {
    int b, head, mt, split, splits, slot;   // slot: of its partial result
    Request q;
};

// The job of workgroup `y` of XCD `x`.  The row tiles of one chunk of keys
// read the same keys: they stay on one XCD, next to each other; the chunks go
// round over the XCDs (workgroups do so by themselves, by their number).
__device__ inline Job job_of(const AttentionArgs& a, const Request& q0, int mt_rows, int c, int x, int y, int lane) {
    Job j{};
    int before = 0, groups_before = 0, partials_before = 0;
    for (int b0 = 0; b0 < a.c.B; b0 += 64) {
        const Request q = b0 ? request_of(a, b0 + lane, mt_rows) : q0;
        const int splits = splits_of(q, c), groups = q.rows ? a.kv.Hkv * splits : 0;
        const int groups_upto = wave_prefix_i32(groups, lane);
        const int first = (x - (groups_before + groups_upto - groups)) & 7;
        const int n = first < groups ? ((groups - first + 7) >> 3) * q.mtiles : 0;
        const int upto = wave_prefix_i32(n, lane);
        const u64 hit = __ballot(before + upto > y);
        const int partials = partials_of(a, q, splits);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            const int local = y - before - __builtin_amdgcn_readlane(upto, at) + __builtin_amdgcn_readlane(n, at);
            j.b = b0 + at;
            j.q.rows = __builtin_amdgcn_readlane(q.rows, at);
            j.q.keys = __builtin_amdgcn_readlane(q.keys, at);
            j.q.mtiles = __builtin_amdgcn_readlane(q.mtiles, at);
            j.q.units = __builtin_amdgcn_readlane(q.units, at);
            j.splits = splits_of(j.q, c);
            j.mt = j.q.mtiles - 1 - local % j.q.mtiles;    // a causal chunk's last rows see most: they go first
            const int g = __builtin_amdgcn_readlane(first, at) + 8 * (local / j.q.mtiles);
            j.split = g % j.splits;
            j.head = g / j.splits;
            j.slot = partials_before + wave_add_i32(lane < at ? partials : 0) +
                     g * j.q.mtiles + j.mt;
            return j;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
        groups_before += __builtin_amdgcn_readlane(groups_upto, 63);
        partials_before += wave_add_i32(partials);
    }
    j.b = -1;
    return j;
}

// ---------------------------------------------------------------------------
// the tile loop
// ---------------------------------------------------------------------------

template <class T>
__device__ inline bool odd_value(uint32_t pair) {          // an infinity or NaN in either half
    constexpr uint32_t e = T::kExponent;
    return (pair & e) == e || (pair & (e << 16)) == (e << 16);
}

// 16 bytes a lane from memory to LDS at `to` + 16 * lane; the waits are the
// caller's: wait_copies<LEFT>() ends when all but the wave's LEFT last copies
// (and loads) have arrived and every LDS read it issued before has its data,
// wait_reads() for the latter alone: then the next copies may overwrite what
// was read.
__device__ inline void copy_to_lds(const uint16_t* from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from),
                 "s"(__builtin_amdgcn_readfirstlane(to)) : "m0");
}
// The same from `base` + `offset` bytes, with a base common to the wave.
__device__ inline void copy_to_lds(const char* base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset),
                 "s"((const char*)uniform((int64_t)base)), "s"(__builtin_amdgcn_readfirstlane(to)) : "m0");
}
template <int LEFT>
__device__ inline void wait_copies() {
    // (loads and copies end in order: all but the LEFT last have)
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LEFT) : "memory");
}
__device__ inline void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

struct True {
    static constexpr bool value = true;
};
struct False {
    static constexpr bool value = false;
};

// What a key and its value are made of: kKey elements, then kRot rotated ones
// that lie elsewhere (kRot = 0: none), and kOut elements of value.
// Heads: keys and values of a head in the cache.
template <int D>
struct Heads {
    static constexpr int kKey = D, kRot = 0, kOut = D;
    static constexpr bool kMade = false;
    static __device__ inline int swizzle_key(int row) { return D == 64 ? (row >> 1) & 7 : row & 15; }
    static __device__ inline int swizzle_out(int row) { return D == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2; }
    static __device__ inline int swizzle_rot(int) { return 0; }
};
// A token's shared rotated part of R elements, 16-byte pieces permuted so that
// a piece of 32 rows spreads over the banks.
template <int R>
struct Rotated {
    static __device__ inline int swizzle_rot(int row) { return R == 64 ? (row >> 1) & 7 : (row >> 2) & 3; }
};
// Expanded: each head's N elements of key and N of value, made from the
// latents, and the rotated part from the cache.
template <int N, int R>
struct Expanded : Rotated<R> {
    static constexpr int kKey = N, kRot = R, kOut = N;
    static constexpr bool kMade = true;
    static __device__ inline int swizzle_key(int row) { return Heads<N>::swizzle_key(row); }
    static __device__ inline int swizzle_out(int row) { return Heads<N>::swizzle_out(row); }
};

template <class T, class L, int WM, int WK, int WD, int KT>
struct Shape {
    static constexpr int kThreads = 64 * WM * WK * WD;
    static constexpr int kMt = WM * kRowsPerWave;
    static constexpr int kKeyTile = KT * L::kKey * 2;      // bytes of a tile of keys, without their rotated part
    static constexpr int kRotTile = KT * L::kRot * 2;
    static constexpr int kTile = kKeyTile + kRotTile;
    static constexpr int kOutTile = KT * L::kOut * 2;
    static constexpr int kGroup = 2 * (kTile + kOutTile);  // the keys' two buffers, the values' two
    static constexpr int kLds = kGroup * WK;
    static constexpr int kPartial = kMt * (L::kOut + 2);   // floats of a split's partial result
};

// One job; every wave of the workgroup calls it.
template <class T, class L, int WM, int WK, int WD, int KT>
__device__ __forceinline__ void attend(const AttentionArgs& a, const Job& job, int c, char* lds, float* partial) {
    using S = Shape<T, L, WM, WK, WD, KT>;
    constexpr int D = L::kKey, kQ = L::kKey + L::kRot, kOut = L::kOut;
    constexpr int NB = KT / 32, KS = kQ / 16, ND = kOut / 32 / WD; // ND: the wave's own blocks of outputs
    constexpr int kUnits16 = D / 8;                        // 16-byte pieces of a key
    constexpr int kRpi = 64 / kUnits16;                    // rows of a wave's copy instruction
    constexpr int kCopies = KT / kRpi / (WM * WD);         // copies of K (and of V) a wave and tile
    constexpr int kPer16 = 16 / kRpi;                      // copies of 16 rows
    static_assert(kCopies * kRpi * WM * WD == KT && kPer16 * kRpi == 16, "whole copies");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wd = wave / WM % WD, wk = wave / (WM * WD), wl = wave % (WM * WD);
    const int half = lane >> 5, col = lane & 31;
    const int b = job.b;
    const int ctx = a.c.ctx_len[b], lead = a.c.lead, nn = job.q.rows - lead;
    const int mrows = job.q.rows * a.G;

    // this lane's query
    const Tiling tiling = tiling_of(mrows, job.q.mtiles);
    const int first_block = job.mt * tiling.base + (job.mt < tiling.more ? job.mt : tiling.more);
    const int blocks = tiling.base + (job.mt < tiling.more);
    const int m0 = (first_block + wm) * kRowsPerWave;
    const int mrow = m0 + col;
    const bool live = wm < blocks && mrow < mrows;
    const int r = live ? mrow / a.G : 0, g = live ? mrow - r * a.G : 0;
    const int64_t row = (int64_t)b * a.c.rows + r;
    const int h = job.head * a.G + g;
    const bool node = a.c.mask && r >= lead;
    const uint32_t* mask = node ? a.c.mask + ((int64_t)b * a.c.n_max + r - lead) * a.c.mask_words : nullptr;
    s16x8 qf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s)
        qf[s] = *(const s16x8*)(a.q + row * a.q_stride + (int64_t)h * kQ + 16 * s + 8 * half);

    // keys below `all` are seen by every query of the wave, keys at or behind
    // `any` by none (64 bits: ctx_len may be anything an int32 holds)
    int64_t all = live ? (int64_t)ctx + (node ? lead : r + 1) : INT64_MAX;
    int64_t any = live ? (int64_t)ctx + (node ? lead + nn : r + 1) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_xor(all, o), y = __shfl_xor(any, o);
        all = x < all ? x : all;
        any = y > any ? y : any;
    }
    all = uniform(all);
    any = uniform(any);
    const bool work = wm < blocks && m0 < mrows;
    const int64_t limit = (int64_t)ctx + r + 1;            // causal rows: first unseen key
    const int64_t first_node = (int64_t)ctx + lead;        // slot of node 0

    // the chunk's tiles, shortened to what the workgroup's rows see
    int last_row = ((first_block + blocks) * kRowsPerWave - 1) / a.G;
    if (last_row > job.q.rows - 1) last_row = job.q.rows - 1;
    int64_t end = (int64_t)ctx + (a.c.mask && last_row >= lead ? job.q.rows : last_row + 1);
    if (end > job.q.keys) end = job.q.keys;
    const int64_t stop = (int64_t)(job.split + 1) * c * kUnit;
    const int k_first = job.split * c * kUnit;
    const int k_end = (int)(end < stop ? end : stop);
    const int tiles = k_end > k_first ? (k_end - k_first + KT - 1) / KT : 0;

    const uint16_t* kbase = a.kv.k + job.head * a.kv.head_stride;
    const uint16_t* vbase = a.kv.v + job.head * a.kv.head_stride;
    const uint16_t* const made = L::kMade ? a.made + ((int64_t)b * a.Hq + job.head) * a.made_keys * (2 * D) : nullptr;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds);
    const uint32_t group = lds0 + wk * S::kGroup;

    // Lane l looks up key l of a tile, one tile before its copies are issued.
    struct Place {
        int page, in;                                      // page id (-1: no such key) and slot in the page
        int tile;                                          // the tile's first key
    };
    const int32_t* table = a.kv.page_table + (int64_t)b * a.kv.max_pages;
    const auto look_up = [&](int t) __attribute__((always_inline)) {
        const int key = k_first + t * KT + (lane & (KT - 1));
        Place p = {-1, 0, k_first + t * KT};
        if (t < tiles && key < k_end) {
            const int i = a.kv.page_shift >= 0 ? key >> a.kv.page_shift : key / a.kv.page_size;
            p.page = table[i];
            p.in = key - i * a.kv.page_size;
        }
        return p;
    };
    const auto is_valid = [&](const Place& p) __attribute__((always_inline)) { return p.page >= 0 && p.page < a.kv.num_pages; };
    // Byte offsets of a lane's copies within the 8 rows they belong to (the
    // permutation of K's pieces repeats after 16).
    constexpr int kOwn = kCopies < kPer16 ? kCopies : kPer16;
    constexpr int kPer8 = kPer16 / 2 < kOwn ? kPer16 / 2 : kOwn;       // a wave's copies of 8 rows
    static_assert(kCopies % kOwn == 0 && kPer16 % kOwn == 0 && kOwn % kPer8 == 0, "whole parts of 8 rows");
    uint32_t koff[kOwn], voff[kOwn];
    const int piece = lane % kUnits16, prow = lane / kUnits16;
    const uint32_t slot_bytes = (uint32_t)(a.kv.slot_stride * 2);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int r16 = (wl * kCopies + i) % kPer16 * kRpi + prow;
        koff[i] = (r16 & 7) * slot_bytes + (piece ^ L::swizzle_key(r16)) * 16;
        voff[i] = (r16 & 7) * slot_bytes + (piece ^ L::swizzle_out(r16)) * 16;
    }
    // Copies of a tile into a buffer of K and of V; a key that is not there
    // comes from some mapped address, its score and value are dropped below.
    const auto issue = [&](const Place& p, int buf) __attribute__((always_inline)) {
        const uint32_t to = group + buf * S::kTile;
        const bool ok = is_valid(p);
        if constexpr (L::kMade) {
            // the rotated parts: pieces of kRotRows rows a copy, the copies dealt to the waves
            constexpr int kRotUnits = L::kRot / 8, kRotRows = 64 / kRotUnits, kRotCopies = KT / kRotRows;
            const int64_t off = ok ? p.page * a.kv.page_stride + p.in * a.kv.slot_stride : 0;
            const int lo = (int)off, hi = (int)(off >> 32);
            const auto offset_of = [&](int trow) __attribute__((always_inline)) {
                return (int64_t)((u64)(uint32_t)__shfl(lo, trow) | (u64)(uint32_t)__shfl(hi, trow) << 32);
            };
#pragma unroll
            for (int i0 = 0; i0 < kRotCopies; i0 += WM * WD) {
                const int at = i0 + wl;
                if (kRotCopies % (WM * WD) != 0 && at >= kRotCopies) break;
                const int trow = at * kRotRows + lane / kRotUnits;
                copy_to_lds(a.kv.v + offset_of(trow) + ((lane % kRotUnits) ^ L::swizzle_rot(trow)) * 8,
                            to + S::kKeyTile + at * 1024);
            }
            // rows of key and value, one after the other; behind the last key the last again
            const int k0 = p.tile;
            const char* const base = (const char*)(made + (int64_t)k0 * (2 * D));
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int at = wl * kCopies + i, trow = at * kRpi + prow;
                const uint32_t r0 = (uint32_t)(k0 + trow < k_end ? trow : k_end - 1 - k0) * (4 * D);
                copy_to_lds(base, r0 + (piece ^ L::swizzle_key(trow)) * 16, to + at * 1024);
                copy_to_lds(base, r0 + 2 * D + (piece ^ L::swizzle_out(trow)) * 16,
                            group + 2 * S::kTile + buf * S::kOutTile + at * 1024);
            }
            return;
        } else if (a.by8) {
            // 8 rows that begin at a multiple of 8 lie in one page: one scalar
            // base for them (three chunks of 779 rows over 11 K keys in pages of
            // 8: 339 us, row by row as below 400)
#pragma unroll
            for (int g = 0; g < kCopies / kPer8; ++g) {
                const int at = wl * kCopies + g * kPer8, row = at * kRpi & ~7;
                const int page = __builtin_amdgcn_readlane(ok ? p.page : 0, row);
                const int in = __builtin_amdgcn_readlane(ok ? p.in : 0, row);
                const int64_t off = page * a.kv.page_stride + in * a.kv.slot_stride;
                const char* const kp = (const char*)(kbase + off);
                const char* const vp = (const char*)(vbase + off);
#pragma unroll
                for (int i = 0; i < kPer8; ++i) {
                    copy_to_lds(kp, koff[(g * kPer8 + i) % kOwn], to + (at + i) * 1024);
                    copy_to_lds(vp, voff[(g * kPer8 + i) % kOwn], to + 2 * S::kTile + (at + i) * 1024);
                }
            }
        } else {
            const int64_t off = ok ? p.page * a.kv.page_stride + p.in * a.kv.slot_stride : 0;
            const int lo = (int)off, hi = (int)(off >> 32);
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int at = wl * kCopies + i, trow = at * kRpi + prow;
                const int64_t o = (int64_t)((u64)(uint32_t)__shfl(lo, trow) | (u64)(uint32_t)__shfl(hi, trow) << 32);
                copy_to_lds(kbase + o + (piece ^ L::swizzle_key(trow)) * 8, to + at * 1024);
                copy_to_lds(vbase + o + (piece ^ L::swizzle_out(trow)) * 8, to + 2 * S::kTile + at * 1024);
            }
        }
    };

    // LDS addresses of this lane's pieces
    // (a permutation changes the low four bits of a piece's number: addresses
    // of 16 pieces and more repeat)
    constexpr int kKeyAddr = D / 16 < 8 ? D / 16 : 8, kRotAddr = L::kRot / 16;
    int kaddr[kKeyAddr], raddr[kRotAddr > 0 ? kRotAddr : 1];
#pragma unroll
    for (int s = 0; s < kKeyAddr; ++s) kaddr[s] = col * D * 2 + ((2 * s + half) ^ L::swizzle_key(col)) * 16;
#pragma unroll
    for (int s = 0; s < kRotAddr; ++s)
        raddr[s] = S::kKeyTile + col * L::kRot * 2 + ((2 * s + half) ^ L::swizzle_rot(col)) * 16;
    const auto key_address = [&](int s) __attribute__((always_inline)) {       // of 16 elements, 8 a lane
        return s < D / 16 ? kaddr[s % kKeyAddr] + s / kKeyAddr * 256 : raddr[s < D / 16 ? 0 : s - D / 16];
    };
    const int vrow = 4 * half + ((lane >> 2) & 3);
    int vaddr[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
        vaddr[d] = vrow * kOut * 2 + ((((wd * ND + d) * 4) ^ L::swizzle_out(vrow)) * 16) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    char* const my = lds + wk * S::kGroup;

    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16{};
    float m = -INFINITY, l = 0;                            // o and l are sums of 2^(score - m), scores in units of log2; l of this lane's keys

    constexpr u64 kFull = KT == 64 ? ~0ull : 0xFFFFFFFFull;
    const auto rescale = [&](float top) __attribute__((always_inline)) {
        const float mm = fmaxf(m, top - lift(T(), top));
        const float w = mm == -INFINITY ? 1.0f : exp2f(m - mm);
        m = mm;
        l *= w;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 16; ++x) o[d][x] *= w;
    };
    const auto value = [&](const char* vt, int d, int x) __attribute__((always_inline)) {  // V^T of 32 elements and 16 keys
        typedef __attribute__((address_space(3))) s16x4 lds4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(vt + vaddr[d] + (16 * x) * kOut * 2));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(vt + vaddr[d] + (16 * x + 8) * kOut * 2));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    // A wave's products go before the other's vector work on the same SIMD
    // (a prompt's chunk 795 -> 769 us).
    const auto scores = [&](const char* kt, int n) __attribute__((always_inline)) {
        f32x16 s = {};
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int x = 0; x < KS; ++x)
            s = mfma(T(), *(const s16x8*)(kt + key_address(x) + n * 32 * (x < D / 16 ? D : L::kRot) * 2), qf[x], s);
        __builtin_amdgcn_s_setprio(0);
        return s;
    };
    // A tile's scores into the sums; `masked` is a type: the tiles that every
    // row sees in full have no code for anything else.
    const auto tile = [&](int k0, f32x16 (&s)[NB], const char* vt, u64 now, auto is_masked) __attribute__((always_inline)) {
        constexpr bool masked = decltype(is_masked)::value;
        uint32_t see[NB];
        if constexpr (masked) {
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int64_t kk = k0 + 32 * n;
                uint32_t w;
                if (!node) {
                    const int64_t left = limit - kk;
                    w = left <= 0 ? 0u : (left >= 32 ? ~0u : (1u << left) - 1);
                } else {
                    const int64_t off = kk - first_node;
                    if (off <= -32) {
                        w = ~0u;
                    } else {
                        const int64_t from = off < 0 ? 0 : off;
                        const int at = (int)(from >> 5), sh = (int)(from & 31);
                        const uint32_t w0 = at < a.c.mask_words ? mask[at] : 0u;
                        const uint32_t w1 = at + 1 < a.c.mask_words ? mask[at + 1] : 0u;
                        w = (uint32_t)(((u64)w1 << 32 | w0) >> sh);
                        const int64_t left = nn - from;
                        w = left <= 0 ? 0u : (left >= 32 ? w : w & ((1u << left) - 1));
                        if (off < 0) w = w << -off | ((1u << -off) - 1);
                    }
                }
                w &= (uint32_t)(now >> (32 * n));
                see[n] = w >> (4 * half);
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    if (!(see[n] >> (8 * (x >> 2) + (x & 3)) & 1)) s[n][x] = -INFINITY;
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int x = 0; x < 16; ++x) top = fmaxf(top, s[n][x]);
        const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
        top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])) * a.scale_log2;
        // m may lag the maximum: most tiles leave o alone.  The weights are
        // rounded to the cache's type for its matrix instruction and summed
        // unrounded (the results' error against 64 bits is 1.3 times what
        // weights in fp32 would leave, most of it their own rounding).
        if (__any(top > m + room(T(), m))) rescale(top);
        const float base = m == -INFINITY ? 0.0f : m;
        s16x8 p[NB * 2];
        float sum = 0;                                     // of the tile: next to a large l its weights are not lost one by one
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][x], a.scale_log2, -base));
                sum += e;
                p[2 * n + (x >> 3)][x & 7] = (short)T::put(e);
            }
        l += sum;
        bool odd = false;
        if constexpr (masked) {
            // An unseen key's weight is 0, but 0 times an infinity or NaN is
            // not: tiles with such values take the careful way.
#pragma unroll 1
            for (int x = 0; x < KT * kOut * 2; x += 1024) {
                const u32x4 v = *(const u32x4*)(vt + x + lane * 16);
                odd |= odd_value<T>(v[0]) || odd_value<T>(v[1]) || odd_value<T>(v[2]) || odd_value<T>(v[3]);
            }
            odd = __any(odd);
        }
        if (!odd) {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int x = 0; x < NB * 2; ++x) o[d] = mfma(T(), value(vt, d, x), p[x], o[d]);
            __builtin_amdgcn_s_setprio(0);
        } else if constexpr (masked) {
            // The finite values are summed as always; whether a query sees
            // an infinity (NaN: of both signs) is counted by two more
            // products, a seen key as 1, or, where its weight is 0, as 256
            // (more than a tile has keys): 0 times an infinity is NaN, as it
            // is in the tiles seen in full.
            static_assert(KT < 256, "a count of ones stays below 256");
            s16x8 seen[NB * 2];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const short one = p[2 * n + (x >> 3)][x & 7] == 0 ? (short)T::k256 : (short)T::kOne;
                    seen[2 * n + (x >> 3)][x & 7] = (see[n] >> (8 * (x >> 2) + (x & 3)) & 1) ? one : (short)0;
                }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                f32x16 up = {}, down = {};
#pragma unroll
                for (int x = 0; x < NB * 2; ++x) {
                    s16x8 v = value(vt, d, x), pos, neg;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const uint32_t bits = (uint16_t)v[y];
                        const bool special = (bits & T::kExponent) == T::kExponent;
                        const bool nan = special && (bits & T::kFraction) != 0;
                        pos[y] = special && (nan || !(bits >> 15)) ? (short)T::kOne : (short)0;
                        neg[y] = special && (nan || (bits >> 15)) ? (short)T::kOne : (short)0;
                        if (special) v[y] = 0;
                    }
                    o[d] = mfma(T(), v, p[x], o[d]);
                    up = mfma(T(), pos, seen[x], up);
                    down = mfma(T(), neg, seen[x], down);
                    __builtin_amdgcn_sched_barrier(0);     // a rare path: registers before speed
                }
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    if (up[x] > 0) o[d][x] += up[x] < 256 ? INFINITY : NAN;
                    if (down[x] > 0) o[d][x] -= down[x] < 256 ? INFINITY : NAN;
                }
            }
        }
    };
    // tiles that every query of the wave sees in full
    const int64_t plain = work ? (all < k_end ? all : k_end) - k_first : 0;
    const int whole = plain > 0 ? (int)(plain / KT) : 0;

    const int rounds = (tiles + WK - 1) / WK;
    const int fast = whole > wk ? (whole - wk + WK - 1) / WK : 0;
    // A wave that has its tiles for itself needs no barrier and fetches two
    // tiles ahead, each into the buffer it has just read; waves that share a
    // tile fetch one ahead, into the buffer that all have left.
    constexpr bool kAlone = WM * WD == 1;
    Place place = look_up(wk);
    u64 valid = __ballot(is_valid(place)), valid1 = 0;     // of this round's tile and of the next
    if (wk < tiles) {
        issue(place, 0);
    }
    place = look_up(wk + WK);
    if constexpr (kAlone) {
        valid1 = __ballot(is_valid(place));
        if (wk + WK < tiles) {
            issue(place, 1);
            place = look_up(wk + 2 * WK);
        }
    }
    const auto round = [&](int i, auto is_masked) __attribute__((always_inline)) {
        const int t = wk + i * WK;
        if constexpr (kAlone) {
            if (t + WK < tiles) wait_copies<2 * kCopies>();
            else wait_copies<0>();
        } else {
            wait_copies<0>();
            __syncthreads();
        }
        const u64 now = valid;
        if constexpr (!kAlone) {
            if (t + WK < tiles) {
                valid = __ballot(is_valid(place));
                issue(place, (i + 1) & 1);
                place = look_up(t + 2 * WK);
            }
        }
        const int k0 = k_first + t * KT;
        bool mine = true;
        if constexpr (decltype(is_masked)::value) mine = work && t < tiles && k0 < any;
        if (mine) {
            f32x16 s[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) s[n] = scores(my + (i & 1) * S::kTile, n);
            tile(k0, s, my + 2 * S::kTile + (i & 1) * S::kOutTile, now, is_masked);
        }
        if constexpr (kAlone) {
            valid = valid1;
            if (t + 2 * WK < tiles) {
                valid1 = __ballot(is_valid(place));
                wait_reads();
                issue(place, i & 1);
                place = look_up(t + 3 * WK);
            }
        }
    };
    int i = 0;
    for (; i < fast && (valid & kFull) == kFull; ++i) round(i, False());
    for (; i < rounds; ++i) round(i, True());
    l += __shfl_xor(l, 32);

    if constexpr (WK > 1) {
        // the key groups' results meet in LDS; group 0 goes on with the sum
        __syncthreads();
        float* const box = (float*)lds;                    // [WK - 1][WM WD][16 ND + 2][64 lanes], a lane's own slots
        constexpr int kSlot = 64;
        const auto at = [&](int k, int x) __attribute__((always_inline)) -> float& { return box[((k * WM * WD + wl) * (16 * ND + 2) + x) * kSlot + lane]; };
        if (wk > 0) {
            at(wk - 1, 0) = m;
            at(wk - 1, 1) = l;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int x = 0; x < 16; ++x) at(wk - 1, 2 + d * 16 + x) = o[d][x];
        }
        __syncthreads();
        if (wk > 0) return;
        float mm = m;
#pragma unroll
        for (int k = 0; k < WK - 1; ++k) mm = fmaxf(mm, at(k, 0));
        const float base = mm == -INFINITY ? 0.0f : mm;
        float w = exp2f(m - base);
        l *= w;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 16; ++x) o[d][x] *= w;
#pragma unroll
        for (int k = 0; k < WK - 1; ++k) {
            const float mk = at(k, 0);
            if (mk == -INFINITY && at(k, 1) == 0) continue;
            w = exp2f(mk - base);
            l += w * at(k, 1);
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int x = 0; x < 16; ++x) o[d][x] += w * at(k, 2 + d * 16 + x);
        }
        m = mm;
    }
    if (!live) return;
    if (job.splits == 1) {
        const float inv = l == 0 ? 0.0f : 1.0f / l;
        uint16_t* const out = a.out + row * a.out_stride + (int64_t)h * kOut + wd * ND * 32 + 4 * half;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s16x4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = (short)T::put(l == 0 ? 0.0f : o[d][4 * x + e] * inv);
                *(s16x4*)(out + d * 32 + 8 * x) = y;
            }
        if (a.lse && half == 0 && wd == 0) a.lse[row * a.Hq + h] = l == 0 ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    } else {
        float* const part = partial + (int64_t)job.slot * S::kPartial;
        const int at = wm * kRowsPerWave + col;
        if (half == 0 && wd == 0) {
            part[at] = m;
            part[S::kMt + at] = l;
        }
        float* const po = part + 2 * S::kMt + (int64_t)at * kOut + wd * ND * 32 + 4 * half;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *(f32x4*)(po + d * 32 + 8 * x) = f32x4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]};
    }
}

// A workgroup a job; those behind the last job end at once.
template <class T, class L, int WM, int WK, int WD, int KT, int PER_CU>
__global__ void __launch_bounds__(64 * WM * WK * WD, (PER_CU * WM * WK * WD + 3) / 4)
    attention_kernel(AttentionArgs a, int slots, int* plan, float* partial) {
    using S = Shape<T, L, WM, WK, WD, KT>;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int lane = threadIdx.x & 63;
    const unsigned id = blockIdx.y * gridDim.x + blockIdx.x;       // (gridDim.x is a multiple of 8)
    const Request q0 = request_of(a, lane, S::kMt);
    const int c = chunk_units(a, q0, S::kMt, slots, lane);
    if (id == 0 && threadIdx.x == 0) *plan = c;            // for combine_kernel
    const Job job = job_of(a, q0, S::kMt, c, (int)(id & 7), (int)(id >> 3), lane);
    if (job.b >= 0) attend<T, L, WM, WK, WD, KT>(a, job, c, lds, partial);
}

// Joins the chunks of split segments: D / 4 lanes for a row and query head (64
// lanes twice the elements for D = 512), a running maximum over its chunks,
// four of which are read at a time.
template <class T, int D, int MT>
__global__ void __launch_bounds__(256) combine_kernel(AttentionArgs a, const int* plan, const float* partial) {
    constexpr int kEach = D > 256 ? D / 256 : 1, kLanes = D / 4 / kEach, kItems = 64 / kLanes;
    const int lane = threadIdx.x & 63;
    const int c = *plan;
    // a wave takes kItems neighbours; the items of a batch of requests are
    // rounded up to whole waves
    int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t before = 0;
    int partials_before = 0;
    for (int b0 = 0; b0 < a.c.B; b0 += 64) {
        const Request mine = request_of(a, b0 + lane, MT);
        const int my_splits = splits_of(mine, c), partials = partials_of(a, mine, my_splits);
        const int n = partials ? mine.rows * a.Hq : 0;     // below 2^31 over the call
        const int upto = wave_prefix_i32(n, lane), partials_upto = wave_prefix_i32(partials, lane);
        const int total = __builtin_amdgcn_readlane(upto, 63);
        const int waves = (total + kItems - 1) / kItems;
        for (; id < before + waves; id += (int64_t)gridDim.x * 4) {
            const int first_item = (int)(id - before) * kItems;
            const bool live = first_item + lane / kLanes < total;
            int local = 0, at = 0;                         // the item, and the lane of its request
#pragma unroll
            for (int i = 0; i < kItems; ++i) {             // with every lane: reads across lanes need them all
                const int it = first_item + i < total ? first_item + i : total - 1;
                const int from = __builtin_ctzll(__ballot(upto > it));
                if (lane / kLanes == i) {
                    local = it;
                    at = from;
                }
            }
            const int b = b0 + at, splits = __shfl(my_splits, at), mtiles = __shfl(mine.mtiles, at);
            const int item = local - __shfl(upto, at) + __shfl(n, at);
            const int r = item / a.Hq, h = item - r * a.Hq;
            const int hk = h / a.G, mrow = r * a.G + (h - hk * a.G), block = mrow / kRowsPerWave;
            const Tiling tiling = tiling_of(__shfl(mine.rows, at) * a.G, mtiles);
            const int long_ones = tiling.more * (tiling.base + 1);     // blocks of the larger tiles
            const int mt = block < long_ones ? block / (tiling.base + 1)
                                             : tiling.more + (block - long_ones) / tiling.base;
            const int first_block = mt * tiling.base + (mt < tiling.more ? mt : tiling.more);
            const int in = mrow - first_block * kRowsPerWave;
            const int64_t first = (int64_t)partials_before + __shfl(partials_upto, at) - __shfl(partials, at) +
                                  (int64_t)hk * splits * mtiles + mt;
            const float* part = partial + first * (MT * (D + 2));
            const int64_t step = (int64_t)mtiles * (MT * (D + 2));
            const int d = lane % kLanes * 4;
            float m = -INFINITY, l = 0;
            f32x4 o[kEach] = {};
            for (int s0 = 0; s0 < splits; s0 += 4) {
                float ms[4], ls[4];
                f32x4 os[4][kEach];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float* p = part + (s0 + i < splits ? s0 + i : s0) * step;
                    ms[i] = p[in];
                    ls[i] = s0 + i < splits ? p[MT + in] : 0.0f;
#pragma unroll
                    for (int x = 0; x < kEach; ++x) os[i][x] = *(const f32x4*)(p + 2 * MT + (int64_t)in * D + x * 256 + d);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (ls[i] == 0) continue;              // nothing seen: its sums are zeros (and m may be -inf)
                    const float mm = fmaxf(m, ms[i]);
                    const float base = mm == -INFINITY ? 0.0f : mm;
                    const float w = exp2f(m - base), v = exp2f(ms[i] - base);
                    m = mm;
                    l = l * w + ls[i] * v;
                    // (m = -inf: o is 0, and so is w)
#pragma unroll
                    for (int x = 0; x < kEach; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[x][e] = o[x][e] * w + os[i][x][e] * v;
                }
            }
            if (!live) continue;
            const float inv = l == 0 ? 0.0f : 1.0f / l;
            const int64_t row = (int64_t)b * a.c.rows + r;
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                s16x4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = (short)T::put(l == 0 ? 0.0f : o[x][e] * inv);
                *(s16x4*)(a.out + row * a.out_stride + (int64_t)h * D + x * 256 + d) = y;
            }
            if (a.lse && d == 0) a.lse[row * a.Hq + h] = l == 0 ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        }
        before += waves;
        partials_before += __builtin_amdgcn_readlane(partials_upto, 63);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int kCus = 256;
constexpr int64_t kMaxGridX = 1 << 20;     // threads along x count in 32 bits
constexpr int kPlanBytes = 256;    // of the workspace: the chunk's size

// Upper bound of a call's jobs on one XCD.  chunk_units() makes at most
// segments + 4 slots chunks, at most `slots` of few segments in one round, and
// none but a segment's last below kMinUnits; a request's groups go round over
// the XCDs, so one XCD has at most an eighth of its chunks and one group of
// mtiles more.
int64_t max_jobs(const AttentionArgs& a, int mt, int slots) {
    const int64_t mtiles = ((int64_t)a.c.rows * a.G + mt - 1) / mt, segments = (int64_t)a.c.B * a.kv.Hkv * mtiles;
    const int64_t units = ((int64_t)a.kv.cap + kUnit - 1) / kUnit;
    int64_t jobs = segments + 4 * slots;
    const int64_t finest = segments * ((units + kMinUnits - 1) / kMinUnits);
    if (finest < jobs) jobs = finest;
    return (jobs + 7) / 8 + a.c.B * mtiles;
}

// The kernel and the join: row tiles of MT rows, results of D elements, `slots`
// workgroups resident at a time.
template <class T, int D, int MT, class Kernel>
hipError_t run_kernel(Kernel kernel, const AttentionArgs& a, int threads, int lds, int slots, void* workspace,
                      hipStream_t stream) {
    const int64_t jobs = 8 * max_jobs(a, MT, slots);
    const int64_t x = jobs < kMaxGridX ? jobs : kMaxGridX;
    int* const plan = (int*)workspace;
    float* const partial = (float*)((char*)workspace + kPlanBytes);
    kernel<<<dim3((unsigned)x, (unsigned)((jobs + x - 1) / x)), threads, lds, stream>>>(a, slots, plan, partial);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t waves = ((int64_t)a.c.B * a.c.rows * a.Hq * (D <= 256 ? D / 4 : 64) + 63) / 64;
    const unsigned groups = waves < 4 * 8 * kCus ? (unsigned)((waves + 3) / 4) : 8 * kCus;
    combine_kernel<T, D, MT><<<groups, 256, 0, stream>>>(a, plan, partial);
    return hipGetLastError();
}

template <class T, class L, int WM, int WK, int WD, int KT, int PER_CU>
hipError_t run(const AttentionArgs& a, int slots, void* workspace, hipStream_t stream) {
    using S = Shape<T, L, WM, WK, WD, KT>;
    return run_kernel<T, L::kOut, S::kMt>(attention_kernel<T, L, WM, WK, WD, KT, PER_CU>, a, S::kThreads, S::kLds, slots,
                                          workspace, stream);
}

// Bytes of the partial results and the plan.  partials_of(): at most work / c
// <= 4 slots of them and one a split segment, of which there are at most work /
// c, too.
size_t partial_bytes(int64_t segments, int slots, int mt, int out) {
    const int64_t partials = 4 * slots + (segments < 4 * slots ? segments : 4 * slots);
    return (size_t)partials * mt * (out + 2) * sizeof(float) + kPlanBytes;
}

}  // namespace
}  // namespace dt
