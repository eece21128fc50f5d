// The absorbed form's tile loop (latent.hip): attention of query rows of C + R
// elements over tokens of C + R elements whose first C are their value, too.
#pragma once

#include "attention_dev.h"

namespace dt {
namespace {

__device__ inline f32x4 mfma16(Bf16, s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, a), __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
}
__device__ inline f32x4 mfma16(F16, s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8, a), __builtin_bit_cast(h16x8, b), c, 0, 0, 0);
}

// Latents: C elements that are key and value of every head, then the rotated
// part.  One tile serves both products, so one permutation has to: pieces move
// by the row's number with its two pairs of bits swapped.  16 consecutive rows
// have 16 different ones (a piece of each row at once, for scores), and rows 4 n
// to 4 n + 3 move their 64-byte groups apart (a group of 4 rows at once, for
// the transposing read).
template <int C, int R>
struct Latents : Rotated<R> {
    static constexpr int kKey = C, kRot = R;
    static __device__ inline int swizzle_key(int row) { return (row & 3) << 2 | ((row >> 2) & 3); }
};

// A workgroup takes 64 rows, a wave 32 of them with half of the work: the
// scores of 16 of a tile's 32 keys, and half of the outputs' elements.  A wave
// with 32 rows for itself would need 144 registers of queries and 256 of
// outputs (C = 512), all of the accumulators and more; this way it is 144 and
// 128, and no product is made twice.  The two waves of a row meet in the tile's
// weights, which go through LDS.
//
// Scores are made transposed, K q^T on 16x16x32 instructions, so that a lane has
// four keys of each of two rows.  The weights lie in LDS as [row][key], the right
// operand of V^T p^T on 32x32x16 instructions; V^T comes from the same tile by
// the transposing read.
//
// A round makes the scores and weights of tile t + 1 and the products of tile t,
// between two barriers, with the copies of the tiles after that in flight.
//
// Measured (C = 512, R = 64, bf16, 64 requests over 33-16383 keys, 0.6 GB): one
// token of 16 heads 151 us, 4.0 TB/s (a copy, read and written, 4.9); of 128
// heads 235 us, 624 TFLOP/s, where memory alone would take 127 and the matrix
// cores 104.  What bounds the latter is one wave a SIMD: a round takes about 3000
// cycles, 1088 of them the matrix core's, the rest the latencies and the issue
// of a wave that nothing else covers.  Trees of 64 nodes, 28 heads, C = 256 over
// 6-10 K keys 206 us, 580 TFLOP/s.  Tried and dropped: eight waves with 64 keys a
// tile (one token of one request 22 us instead of 24, 128 heads 285, trees 282);
// all 64 rows and a quarter of the outputs a wave (half of the LDS reads of the
// second product; 128 heads 252 where this took 254: it is not those reads).
template <int C, int R>
struct Latent {
    static constexpr int kKeys = 32, kRows = 64;
    static constexpr int kBuffers = C == 512 ? 4 : 3;      // C = 256: two workgroups on a compute unit
    static constexpr int kPerCu = C == 512 ? 1 : 2;
    static constexpr int kKeyTile = kKeys * C * 2, kTile = kKeyTile + kKeys * R * 2;
    static constexpr int kWeightRow = 80;                  // bytes of a row of weights: 64, spread over the banks
    static constexpr int kWeights = kBuffers * kTile;      // where the weights' two buffers begin
    static constexpr int kMaxima = kWeights + 2 * kRows * kWeightRow;      // [2][2 waves][rows] floats
    static constexpr int kOdd = kMaxima + 2 * 2 * kRows * 4;               // [4] words
    static constexpr int kThere = kOdd + 16;                               // [2][up to 64 tiles][4 waves] bytes
    static constexpr int kLds = kThere + 512;
    static constexpr int kPartial = kRows * (C + 2);       // floats of a split's partial result
    static_assert(kLds * kPerCu <= 160 * 1024, "LDS of a compute unit");
};

template <class T, int C, int R, bool BY8>
__device__ __forceinline__ void attend_latents(const AttentionArgs& a, const Job& job, int c, char* lds, float* partial) {
    using L = Latents<C, R>;
    using S = Latent<C, R>;
    constexpr int kQ = C + R, KS = kQ / 32, ND = C / 64;   // ND: blocks of 32 outputs of the wave
    constexpr int kPieces = C / 8, kRpc = 64 / kPieces;    // 16-byte pieces of a latent, rows of a copy
    constexpr int kCopies = 8 / kRpc + 1;                  // of a wave and tile: 8 rows, and their rotated parts
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wr = wave & 1, wd = wave >> 1;
    const int quad = lane >> 4, col = lane & 15, half = lane >> 5, row32 = lane & 31;
    const int b = job.b;
    const int ctx = a.c.ctx_len[b], lead = a.c.lead, nn = job.q.rows - lead;
    const int mrows = job.q.rows * a.Hq;

    const Tiling tiling = tiling_of(mrows, job.q.mtiles);
    const int first_block = job.mt * tiling.base + (job.mt < tiling.more ? job.mt : tiling.more);
    const int blocks = tiling.base + (job.mt < tiling.more);
    const int m0 = (first_block + wr) * kRowsPerWave;

    // the rows whose scores this lane holds
    int chunk_row[2];
    s16x8 qf[KS][2];
    // of step 4 n + i a lane takes piece 16 n + 4 quad + i: eight lanes of four
    // rows and two quads, as the LDS reads them at once, lie in different banks
    const auto element = [&](int s) __attribute__((always_inline)) {
        return s < C / 32 ? (s / 4 * 16 + 4 * quad + s % 4) * 8 : C + (4 * (s - C / 32) + quad) * 8;
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int mrow = m0 + 16 * i + col;
        const bool live = wr < blocks && mrow < mrows;
        const int r = live ? mrow / a.Hq : 0, h = live ? mrow - r * a.Hq : 0;
        const int64_t row = (int64_t)b * a.c.rows + r;
        chunk_row[i] = r;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s][i] = *(const s16x8*)(a.q + row * a.q_stride + (int64_t)h * kQ + element(s));
    }

    // the tiles of the workgroup's rows, and how many of them every row sees in full
    const int row0 = first_block * kRowsPerWave / a.Hq;
    int row1 = ((first_block + blocks) * kRowsPerWave - 1) / a.Hq;
    if (row1 > job.q.rows - 1) row1 = job.q.rows - 1;
    int64_t end = (int64_t)ctx + (a.c.mask && row1 >= lead ? job.q.rows : row1 + 1);
    if (end > job.q.keys) end = job.q.keys;
    const int64_t stop = (int64_t)(job.split + 1) * c * kUnit;
    const int k_first = job.split * c * kUnit;
    const int k_end = (int)(end < stop ? end : stop);
    const int tiles = k_end > k_first ? (k_end - k_first + S::kKeys - 1) / S::kKeys : 0;
    int64_t all = (int64_t)ctx + (a.c.mask && row0 >= lead ? lead : row0 + 1);
    if (all > k_end) all = k_end;
    const int whole = all > k_first ? (int)((all - k_first) / S::kKeys) : 0;

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds);

    // Where the wave's eight keys of a tile lie.  Eight keys that begin at a
    // multiple of 8 lie in one page (BY8): a lane holds this for one of 64 tiles.
    // Otherwise it does so for one key of 8 tiles.  The bytes in LDS say which keys
    // are there; behind the last key the offset is the last one's.  (An entry a
    // round, by a scalar load, made every round wait for it.)
    constexpr int kNoLoads = 0x0F70;                       // s_waitcnt's vmcnt(0)
    constexpr int kWindow = BY8 ? 64 : 8;
    uint32_t off_lo = 0, off_hi = 0;
    const auto look_up = [&](int window) __attribute__((always_inline)) {
        const int k0 = k_first + (window * kWindow + (BY8 ? lane : lane >> 3)) * S::kKeys + 8 * wave;
        const int own = BY8 ? k0 : k0 + (lane & 7), last = BY8 ? (k_end - 1) & ~7 : k_end - 1, key = own < last ? own : last;
        const int at = (int)((uint64_t)(uint32_t)key * a.page_mul >> a.page_rsh);
        const int page = a.kv.page_table[(int64_t)b * a.kv.max_pages + at];
        const bool there = page >= 0 && page < a.kv.num_pages;
        const int64_t off = there ? page * a.kv.page_stride + (key - at * a.kv.page_size) * a.kv.slot_stride : 0;
        off_lo = (uint32_t)off;
        off_hi = (uint32_t)(off >> 32);
        uint8_t* const to = (uint8_t*)(lds + S::kThere + (window & 1) * 256) + wave;
        if constexpr (BY8) {
            const int left = k_end - k0;                   // of the wave's keys
            const uint32_t valid = left >= 8 ? 0xFFu : (left <= 0 ? 0u : (1u << left) - 1);
            to[4 * lane] = there ? (uint8_t)valid : 0;     // (the last page's slots behind the last key are the cache's own)
        } else {
            const u64 valid = __ballot(there && own < k_end);
            if ((lane & 7) == 0) to[4 * (lane >> 3)] = (uint8_t)(valid >> lane);
        }
    };
    const auto there_of = [&](int t) __attribute__((always_inline)) {
        return ((const uint32_t*)(lds + S::kThere))[(t / kWindow & 1) * 64 + t % kWindow];
    };
    // The copies of a tile: rows 8 wave .. 8 wave + 7; a key that is not there
    // comes from the first slot (of its page), its score is dropped below.  They
    // are issued one by one, between other work: the unit that takes them needs 16
    // cycles each, and holds up a wave that issues them in a row.
    constexpr int kRotPieces = R / 8;
    const uint32_t slot_bytes = (uint32_t)(a.kv.slot_stride * 2);
    const int rot_row = lane / kRotPieces & 7, rot_piece = (lane % kRotPieces) ^ L::swizzle_rot(wave * 8 + rot_row);
    struct Copies {
        const char* base;                                  // BY8: of the wave's keys
        int in;                                            // else where in the window the tile is
        uint32_t to;
    };
    const auto begin_copies = [&](int t, int buf) __attribute__((always_inline)) {
        Copies c{};
        c.to = lds0 + buf * S::kTile;
        c.in = t % kWindow;
        if constexpr (BY8) {
            const uint32_t lo = __builtin_amdgcn_readlane(off_lo, c.in), hi = __builtin_amdgcn_readlane(off_hi, c.in);
            c.base = (const char*)(a.kv.k + (int64_t)((u64)hi << 32 | lo));
        }
        return c;
    };
    const auto copy = [&](const Copies& c, int i) __attribute__((always_inline)) {
        const bool rot = i == kCopies - 1;
        const int at = wave * (kCopies - 1) + i, row8 = rot ? rot_row : i * kRpc + lane / kPieces;
        const uint32_t piece = (lane % kPieces) ^ L::swizzle_key(wave * 8 + row8);
        const uint32_t to = rot ? c.to + S::kKeyTile + wave * 8 * R * 2 : c.to + at * 1024;
        if constexpr (BY8) {
            if (!rot) copy_to_lds(c.base, row8 * slot_bytes + piece * 16, to);
            else if (lane < 8 * kRotPieces) copy_to_lds(c.base + C * 2, rot_row * slot_bytes + rot_piece * 16, to);
        } else {
            const int from = 8 * c.in + row8;
            const int64_t o = (int64_t)((u64)(uint32_t)__shfl((int)off_lo, from) | (u64)(uint32_t)__shfl((int)off_hi, from) << 32);
            if (!rot) copy_to_lds(a.kv.k + o + piece * 8, to);
            else if (lane < 8 * kRotPieces) copy_to_lds(a.kv.v + o + rot_piece * 8, to);
        }
    };

    // LDS addresses of this lane's pieces within a tile
    const int krow = 16 * wd + col;
    int kaddr[4], raddr[R / 32];                           // (a permutation changes the low four bits of a piece's number)
#pragma unroll
    for (int s = 0; s < 4; ++s) kaddr[s] = krow * C * 2 + ((4 * quad + s) ^ L::swizzle_key(krow)) * 16;
#pragma unroll
    for (int s = 0; s < R / 32; ++s) raddr[s] = S::kKeyTile + krow * R * 2 + ((4 * s + quad) ^ L::swizzle_rot(krow)) * 16;
    int vaddr[4], vaddr4[4];                               // of keys 8 half .. + 3, and of the next four
    {
        const int in = ((lane >> 4) & 1) * 32 + (lane & 3) * 8, vrow = 8 * half + ((lane >> 2) & 3);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int at = wd * (C / 2) * 2 + d * 64 + in;
            vaddr[d] = vrow * C * 2 + (at ^ (L::swizzle_key(vrow) * 16));
            vaddr4[d] = (vrow + 4) * C * 2 + (at ^ (L::swizzle_key(vrow + 4) * 16));
        }
    }
    const auto value = [&](const char* vt, int d, int x) __attribute__((always_inline)) {      // V^T of 32 elements and 16 keys
        typedef __attribute__((address_space(3))) s16x4 lds4;
        const int at = d / 4 * 256 + 16 * x * C * 2;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(vt + vaddr[d % 4] + at));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(vt + vaddr4[d % 4] + at));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    char* const weights = lds + S::kWeights + wr * 32 * S::kWeightRow;     // this wave's rows in the first buffer
    float* const maxima = (float*)(lds + S::kMaxima) + wr * 32;
    const auto max_of = [&](int buf, int d, int row) __attribute__((always_inline)) -> float& {
        return maxima[(buf * 2 + d) * S::kRows + row];
    };

    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16{};
    float m_out = -INFINITY;                               // what row32's outputs are relative to (units of log2)
    // the same for the scores' rows, as it is taken from scores, and from where on
    // it is raised; sums of this lane's keys
    float m[2] = {-INFINITY, -INFINITY}, base[2] = {0, 0}, limit[2] = {-INFINITY, -INFINITY}, l[2] = {0, 0};
    const auto factor = [](float from, float to) __attribute__((always_inline)) {      // 2^(from - to), from <= to
        return to == -INFINITY ? 1.0f : exp2f(from - to);
    };

    // A tile's scores, with some of another tile's copies between them.  The keys are read
    // kAhead steps (of 32 cycles) before their products.  The order is held as
    // written: left to itself the compiler saves registers and waits for each read
    // (64 requests' tokens of 128 heads: 290 us).
    constexpr int kEarly = (KS + 3) / 4 < kCopies ? (KS + 3) / 4 : kCopies;
    const auto scores = [&](const char* kt, f32x4 (&s)[2], const Copies& c) __attribute__((always_inline)) {
        constexpr int kAhead = 6;
        const auto key = [&](int x) __attribute__((always_inline)) {
            return *(const s16x8*)(kt + (x < C / 32 ? kaddr[x % 4] + x / 4 * 256 : raddr[x < C / 32 ? 0 : x - C / 32]));
        };
        s16x8 k[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) k[x] = key(x);
        f32x4 part[2][2] = {};                             // (of even and odd steps: a product a chain is under way)
#pragma unroll
        for (int x = 0; x < KS; ++x) {
#pragma unroll
            for (int i = 0; i < 2; ++i) part[x % 2][i] = mfma16(T(), k[x % kAhead], qf[x][i], part[x % 2][i]);
            __builtin_amdgcn_sched_barrier(0);
            if (x + kAhead < KS) k[x % kAhead] = key(x + kAhead);
            if (x % 4 == 0 && x / 4 < kEarly) copy(c, x / 4);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) s[i] = part[0][i] + part[1][i];
    };
    // Which of the 32 keys from k0 on chunk row r sees.
    const auto see_bits = [&](int r, int k0) __attribute__((always_inline)) {
        if (!a.c.mask || r < lead) {
            const int64_t left = (int64_t)ctx + r + 1 - k0;
            return left <= 0 ? 0u : (left >= 32 ? ~0u : (1u << left) - 1);
        }
        const int64_t off = (int64_t)k0 - ctx - lead;      // of the first key, as a node's number
        if (off <= -32) return ~0u;
        const uint32_t* const mask = a.c.mask + ((int64_t)b * a.c.n_max + r - lead) * a.c.mask_words;
        const int64_t from = off < 0 ? 0 : off;
        const int at = (int)(from >> 5), sh = (int)(from & 31);
        const uint32_t w0 = at < a.c.mask_words ? mask[at] : 0u;
        const uint32_t w1 = at + 1 < a.c.mask_words ? mask[at + 1] : 0u;
        uint32_t w = (uint32_t)(((u64)w1 << 32 | w0) >> sh);
        const int64_t left = nn - from;
        w = left <= 0 ? 0u : (left >= 32 ? w : w & ((1u << left) - 1));
        if (off < 0) w = w << -off | ((1u << -off) - 1);
        return w;
    };
    // What a row's weights are relative to lags behind its largest score, so that a
    // tile of ordinary scores needs no maximum over lanes and no branch: a lane's
    // four scores are compared with the limit, and where one passes it, in any
    // row of the wave, the rows' largest scores take their place.
    const auto top_of = [&](const f32x4& s) __attribute__((always_inline)) {
        return fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])) * a.scale_log2;
    };
    const auto set = [&](int i, float to) __attribute__((always_inline)) {
        m[i] = to;
        base[i] = to == -INFINITY ? 0.0f : to;
        limit[i] = to + room(T(), to);
    };
    const auto raise = [&](const f32x4 (&s)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float top = top_of(s[i]);
            const auto p16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(top), __float_as_uint(top), false, false);
            top = fmaxf(__uint_as_float(p16[0]), __uint_as_float(p16[1]));
            const auto p32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
            top = fmaxf(__uint_as_float(p32[0]), __uint_as_float(p32[1]));
            const float to = top > limit[i] ? fmaxf(m[i], top - lift(T(), top)) : m[i];
            l[i] *= factor(m[i], to);
            set(i, to);
        }
    };
    // Scores into weights, in kParts parts that stand between products.  The
    // weights are rounded to the cache's type for the second product and summed
    // unrounded.
    constexpr int kParts = 12;
    const auto weigh = [&](int part, f32x4 (&s)[2], int buf) __attribute__((always_inline)) {
        const int i = part & 1, x = part >> 1, row = 16 * i + col;
        if (part < 8) {
            s[i][x] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][x], a.scale_log2, -base[i]));
        } else if (part < 10) {
            l[i] += (s[i][0] + s[i][1]) + (s[i][2] + s[i][3]);
            max_of(buf, wd, row) = m[i];                   // (by four lanes)
        } else {
            s16x4 p;
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = (short)T::put(s[i][e]);
            *(s16x4*)(weights + buf * S::kRows * S::kWeightRow + row * S::kWeightRow + 32 * wd + 8 * quad) = p;
        }
    };
    // Tile t's weights, and what they are relative to, as the row's two waves made them.
    struct Met {
        s16x8 p[2];
        float m0, m1;
    };
    const auto meet = [&](int buf) __attribute__((always_inline)) {
        const char* const at = weights + buf * S::kRows * S::kWeightRow + row32 * S::kWeightRow + 16 * half;
        return Met{{*(const s16x8*)at, *(const s16x8*)(at + 32)}, max_of(buf, 0, row32), max_of(buf, 1, row32)};
    };
    // That becomes one, the larger: for this wave's sums and outputs, and the
    // weights as read.  Weights of the wave that was behind are rounded a second
    // time, in those tiles only: they are off by two half steps of the type at most.
    // One rounding would take weights of 32 bits through LDS in every tile.
    const auto agree = [&](int buf, Met& met) __attribute__((always_inline)) {
        s16x8 (&p)[2] = met.p;
        const float m0 = met.m0, m1 = met.m1, mm = fmaxf(m0, m1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float both = fmaxf(max_of(buf, 0, 16 * i + col), max_of(buf, 1, 16 * i + col));
            l[i] *= factor(m[i], both);
            set(i, both);
        }
        const float w = factor(m_out, mm);
        m_out = mm;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            // (an accumulator at a time through vector registers: the queries need the others)
            if constexpr (S::kPerCu == 1) asm volatile("" : "+a"(o[d]));
#pragma unroll
            for (int x = 0; x < 16; ++x) o[d][x] *= w;
            if constexpr (S::kPerCu == 1) asm volatile("" : "+a"(o[d]));
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float f = factor(x ? m1 : m0, mm);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[x][e] = (short)T::put(T::get((uint16_t)p[x][e]) * f);
        }
    };
    // Tile t's products, with the next tile's weights made between them (`weighs`
    // is a type).  Neighbours are products of different sums: none waits for the
    // one before.  Values are read kAhead products before theirs, in this order.
    const auto products = [&](const char* vt, const s16x8 (&p)[2], f32x4 (&s)[2], int buf, const Copies& c, auto weighs) __attribute__((always_inline)) {
        constexpr int kAhead = 4, kSteps = 2 * ND, kEach = (kParts + kSteps - 1) / kSteps, kEvery = kSteps / (kCopies - kEarly + 1);
        static_assert(kEvery > 0, "a step for each copy");
        s16x8 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = value(vt, i % ND, i / ND);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            o[i % ND] = mfma(T(), v[i % kAhead], p[i / ND], o[i % ND]);
            __builtin_amdgcn_sched_barrier(0);
            if (i + kAhead < kSteps) v[i % kAhead] = value(vt, (i + kAhead) % ND, (i + kAhead) / ND);
            if constexpr (decltype(weighs)::value) {
#pragma unroll
                for (int part = i * kEach; part < (i + 1) * kEach && part < kParts; ++part) weigh(part, s, buf);
                if (i % kEvery == kEvery - 1 && kEarly + i / kEvery < kCopies) copy(c, kEarly + i / kEvery);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    int buf = S::kBuffers - 1;                             // of tile t; t + 1 has the next one
    const auto next = [](int i) __attribute__((always_inline)) { return i + 1 == S::kBuffers ? 0 : i + 1; };
    // tile t's products and tile t + 1's weights
    const auto round = [&](int t, auto is_started) __attribute__((always_inline)) {
        constexpr bool started = decltype(is_started)::value;
        wait_copies<(S::kBuffers - 3) * kCopies>();
        __syncthreads();
        const int b1 = next(buf), before = buf == 0 ? S::kBuffers - 1 : buf - 1;
        Met met{};
        if (started) met = meet(t & 1);
        // into the buffer that tile t - 1 has left; behind the last tile, what nobody
        // reads: every round has as many copies
        const int ahead = t + S::kBuffers - 1;
        if (__builtin_expect(ahead % kWindow == 0, 0)) look_up(ahead / kWindow);
        const Copies c = begin_copies(ahead, before);
        const uint32_t flags = there_of(t + 1);
        f32x4 s[2];
        scores(lds + b1 * S::kTile, s, c);
        const uint32_t now = (uint32_t)__builtin_amdgcn_readfirstlane((int)flags);
        // (one branch for all that a tile may need besides; __any's value is the wave's)
        const bool masked = t + 1 >= whole || now != ~0u;
        const bool moved = (met.m0 != met.m1) | (met.m0 > m_out) | (top_of(s[0]) > limit[0]) | (top_of(s[1]) > limit[1]);
        if (__builtin_expect(masked || __any(moved), 0)) {
            if (masked) {
                // A row's weight for a key it does not see is 0, but 0 times an
                // infinity or NaN is not: latents with such elements are found,
                // rows that see them become NaN, and the elements 0 (the scores
                // of all waves have been made by then).
                char* const tile = lds + b1 * S::kTile;
                uint32_t odd = 0;
#pragma unroll 1
                for (int i = 0; i < 8; i += kRpc) {
                    const u32x4 v = *(const u32x4*)(tile + (wave * 8 + i) * C * 2 + lane * 16);
                    const u64 hit = __ballot(odd_value<T>(v[0]) || odd_value<T>(v[1]) || odd_value<T>(v[2]) || odd_value<T>(v[3]));
                    if (kRpc == 1) odd |= (hit != 0 ? 1u : 0u) << i;
                    else odd |= ((uint32_t)hit != 0 ? 1u : 0u) << i | (hit >> 32 != 0 ? 2u : 0u) << i;
                }
                uint32_t* const odds = (uint32_t*)(lds + S::kOdd);
                if (lane == 0) odds[wave] = odd;
                __syncthreads();
                const uint32_t any_odd = odds[0] | odds[1] << 8 | odds[2] << 16 | odds[3] << 24;
                if (odd) {
#pragma unroll 1
                    for (int i = 0; i < 8; i += kRpc) {
                        uint16_t* const v = (uint16_t*)(tile + (wave * 8 + i) * C * 2 + lane * 16);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if ((v[e] & T::kExponent) == T::kExponent) v[e] = 0;
                    }
                }
                const int k0 = k_first + (t + 1) * S::kKeys;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t see = see_bits(chunk_row[i], k0) & now;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int key = 16 * wd + 4 * quad + x;
                        if (!(see >> key & 1)) s[i][x] = -INFINITY;
                        else if (any_odd >> key & 1) s[i][x] = NAN;
                    }
                }
                // The loads of the mask end here: a path on which the compiler takes
                // one to be under way has it wait for all copies behind this block, in
                // every round (1100 cycles of 4000).
                __builtin_amdgcn_s_waitcnt(kNoLoads);
            }
            if (started) agree(t & 1, met);
            raise(s);
        }
        if constexpr (started) {
            products(lds + buf * S::kTile, met.p, s, (t + 1) & 1, c, True());
        } else {
#pragma unroll
            for (int i = kEarly; i < kCopies; ++i) copy(c, i);
#pragma unroll
            for (int i = 0; i < kParts; ++i) weigh(i, s, (t + 1) & 1);
        }
        buf = b1;
    };
    if (tiles > 0) {
        look_up(0);
#pragma unroll
        for (int i = 0; i < S::kBuffers - 2; ++i) {
            const Copies c = begin_copies(i, i);
#pragma unroll
            for (int x = 0; x < kCopies; ++x) copy(c, x);
        }
        round(-1, False());
        for (int t = 0; t + 1 < tiles; ++t) round(t, True());
        // the last tile's products
        wait_copies<0>();
        __syncthreads();
        Met met = meet((tiles - 1) & 1);
        agree((tiles - 1) & 1, met);
        f32x4 none[2] = {};
        products(lds + buf * S::kTile, met.p, none, 0, Copies{}, False());
    }
    // the sums of a row's weights: of the lanes, then of the two waves
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor(l[i], 16);
        l[i] += __shfl_xor(l[i], 32);
    }
    __syncthreads();
    if (quad == 0) {
        max_of(0, wd, col) = l[0];
        max_of(0, wd, 16 + col) = l[1];
    }
    __syncthreads();
    const float total = max_of(0, 0, row32) + max_of(0, 1, row32);
    const int mrow = m0 + row32;
    if (wr >= blocks || mrow >= mrows) return;
    const int r = mrow / a.Hq, h = mrow - r * a.Hq;
    const int64_t row = (int64_t)b * a.c.rows + r;
    if (job.splits == 1) {
        const float inv = total == 0 ? 0.0f : 1.0f / total;
        uint16_t* const out = a.out + row * a.out_stride + (int64_t)h * C + wd * (C / 2) + 4 * half;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s16x4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = (short)T::put(total == 0 ? 0.0f : o[d][4 * x + e] * inv);
                *(s16x4*)(out + d * 32 + 8 * x) = y;
            }
        if (a.lse && half == 0 && wd == 0)
            a.lse[row * a.Hq + h] = total == 0 ? -INFINITY : (m_out + log2f(total)) * 0.69314718055994531f;
    } else {
        float* const part = partial + (int64_t)job.slot * S::kPartial;
        const int at = wr * 32 + row32;
        if (half == 0 && wd == 0) {
            part[at] = m_out;
            part[S::kRows + at] = total;
        }
        float* const po = part + 2 * S::kRows + (int64_t)at * C + wd * (C / 2) + 4 * half;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *(f32x4*)(po + d * 32 + 8 * x) = f32x4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]};
    }
}

// A workgroup a job; those behind the last job end at once.
template <class T, int C, int R, bool BY8>
__global__ void __launch_bounds__(256, C == 512 ? 1 : 2) latent_kernel(AttentionArgs a, int slots, int* plan, float* partial) {
    using S = Latent<C, R>;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int lane = threadIdx.x & 63;
    const unsigned id = blockIdx.y * gridDim.x + blockIdx.x;       // (gridDim.x is a multiple of 8)
    const Request q0 = request_of(a, lane, S::kRows);
    const int c = chunk_units(a, q0, S::kRows, slots, lane);
    if (id == 0 && threadIdx.x == 0) *plan = c;            // for combine_kernel
    const Job job = job_of(a, q0, S::kRows, c, (int)(id & 7), (int)(id >> 3), lane);
    if (job.b >= 0) attend_latents<T, C, R, BY8>(a, job, c, lds, partial);
}

}  // namespace
}  // namespace dt
