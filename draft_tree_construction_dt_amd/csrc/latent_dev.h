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
    static constexpr int kLds = kOdd + 16;
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
    struct Query {
        int r;
        bool node;
        const uint32_t* mask;
    } query[2];
    s16x8 qf[KS][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int mrow = m0 + 16 * i + col;
        const bool live = wr < blocks && mrow < mrows;
        const int r = live ? mrow / a.Hq : 0, h = live ? mrow - r * a.Hq : 0;
        const int64_t row = (int64_t)b * a.c.rows + r;
        query[i].r = r;
        query[i].node = a.c.mask && r >= lead;
        query[i].mask = query[i].node ? a.c.mask + ((int64_t)b * a.c.n_max + r - lead) * a.c.mask_words : nullptr;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s][i] = *(const s16x8*)(a.q + row * a.q_stride + (int64_t)h * kQ + 32 * s + 8 * quad);
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

    // Where the keys of a tile lie, a round before their copies are issued.  Eight
    // keys that begin at a multiple of 8 lie in one page (by8): the wave's own, and
    // four a tile to know which are there, read by scalar loads, which the copies'
    // counter does not wait for.  Otherwise lane l looks up key l.
    struct Place {
        int page, in;                                      // of the wave's eight keys (this lane's key)
        int pages[4];                                      // of the tile's, eight each
    };
    typedef const __attribute__((address_space(4))) int32_t* Table;
    const Table table = (Table)(uintptr_t)(a.kv.page_table + (int64_t)b * a.kv.max_pages);
    const auto look_up = [&](int t) __attribute__((always_inline)) {
        Place p = {-1, 0, {-1, -1, -1, -1}};
        if (t >= tiles) return p;
        const int k0 = k_first + t * S::kKeys;
        const auto number = [&](int key) __attribute__((always_inline)) {
            return a.kv.page_shift >= 0 ? key >> a.kv.page_shift : key / a.kv.page_size;
        };
        const int mine = BY8 ? k0 + 8 * wave : k0 + row32;
        if (mine < k_end) {
            const int at = number(mine);
            p.page = table[at];
            p.in = mine - at * a.kv.page_size;
        }
        if constexpr (BY8) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k0 + 8 * i < k_end) p.pages[i] = table[number(k0 + 8 * i)];
        }
        return p;
    };
    const auto there = [&](int page) __attribute__((always_inline)) { return page >= 0 && page < a.kv.num_pages; };
    const auto valid_keys = [&](const Place& p, int t) __attribute__((always_inline)) {
        if constexpr (!BY8) return (uint32_t)__ballot(there(p.page));
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= there(p.pages[i]) ? 0xFFu << (8 * i) : 0u;
        const int left = k_end - (k_first + t * S::kKeys);
        return left >= 32 ? w : (left <= 0 ? 0u : w & ((1u << left) - 1));
    };
    // The copies of a tile: rows 8 wave .. 8 wave + 7; a key that is not there
    // comes from the first slot (of its page), its score is dropped below.
    constexpr int kRotPieces = R / 8;
    const uint32_t slot_bytes = (uint32_t)(a.kv.slot_stride * 2);
    const int rot_row = lane / kRotPieces & 7, rot_piece = (lane % kRotPieces) ^ L::swizzle_rot(wave * 8 + rot_row);
    const auto issue = [&](const Place& p, int buf) __attribute__((always_inline)) {
        const uint32_t to = lds0 + buf * S::kTile, to_rot = to + S::kKeyTile + wave * 8 * R * 2;
        if constexpr (BY8) {
            const int64_t off = there(p.page) ? p.page * a.kv.page_stride + p.in * a.kv.slot_stride : 0;
            // (the last page's slots behind the last key are the cache's own)
            const char* const base = (const char*)(a.kv.k + off);
#pragma unroll
            for (int i = 0; i < kCopies - 1; ++i) {
                const int at = wave * (kCopies - 1) + i, row8 = i * kRpc + lane / kPieces;
                const uint32_t piece = (lane % kPieces) ^ L::swizzle_key(wave * 8 + row8);
                copy_to_lds(base, row8 * slot_bytes + piece * 16, to + at * 1024);
            }
            if (lane < 8 * kRotPieces) copy_to_lds(base + C * 2, rot_row * slot_bytes + rot_piece * 16, to_rot);
        } else {
            const int64_t off = there(p.page) ? p.page * a.kv.page_stride + p.in * a.kv.slot_stride : 0;
            const int lo = (int)off, hi = (int)(off >> 32);
            const auto offset_of = [&](int trow) __attribute__((always_inline)) {
                return (int64_t)((u64)(uint32_t)__shfl(lo, trow) | (u64)(uint32_t)__shfl(hi, trow) << 32);
            };
#pragma unroll
            for (int i = 0; i < kCopies - 1; ++i) {
                const int at = wave * (kCopies - 1) + i, trow = at * kRpc + lane / kPieces;
                copy_to_lds(a.kv.k + offset_of(trow) + ((lane % kPieces) ^ L::swizzle_key(trow)) * 8, to + at * 1024);
            }
            const int64_t o = offset_of(wave * 8 + rot_row);
            if (lane < 8 * kRotPieces) copy_to_lds(a.kv.v + o + rot_piece * 8, to_rot);
        }
    };

    // LDS addresses of this lane's pieces within a tile
    const int krow = 16 * wd + col;
    constexpr int kKeyAddr = 4;                            // the permutation's low four bits repeat after 4 x 32 elements
    int kaddr[kKeyAddr], raddr[R / 32];
#pragma unroll
    for (int s = 0; s < kKeyAddr; ++s) kaddr[s] = krow * C * 2 + ((4 * s + quad) ^ L::swizzle_key(krow)) * 16;
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
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0, 0};    // the same for the scores' rows; sums of this lane's keys
    const auto factor = [](float from, float to) __attribute__((always_inline)) {      // 2^(from - to), from <= to
        return to == -INFINITY ? 1.0f : exp2f(from - to);
    };

    // The tile's scores, then its weights into LDS.
    const auto scores = [&](const char* kt, f32x4 (&s)[2]) __attribute__((always_inline)) {
        s[0] = s[1] = f32x4{};
#pragma unroll
        for (int x = 0; x < KS; ++x) {
            const s16x8 k = *(const s16x8*)(kt + (x < C / 32 ? kaddr[x % 4] + x / 4 * 256 : raddr[x < C / 32 ? 0 : x - C / 32]));
#pragma unroll
            for (int i = 0; i < 2; ++i) s[i] = mfma16(T(), k, qf[x][i], s[i]);
        }
        // a few pieces ahead, no more: the queries need the registers
        constexpr int kAhead = 6;
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int x = 0; x < KS - kAhead; ++x) {
            __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 2 * kAhead, 0);
    };
    const auto see_bits = [&](const Query& q, int k0) __attribute__((always_inline)) {
        if (!q.node) {
            const int64_t left = (int64_t)ctx + q.r + 1 - k0;
            return left <= 0 ? 0u : (left >= 32 ? ~0u : (1u << left) - 1);
        }
        const int64_t off = (int64_t)k0 - ctx - lead;      // of the tile's first key, as a node's number
        if (off <= -32) return ~0u;
        const int64_t from = off < 0 ? 0 : off;
        const int at = (int)(from >> 5), sh = (int)(from & 31);
        const uint32_t w0 = at < a.c.mask_words ? q.mask[at] : 0u;
        const uint32_t w1 = at + 1 < a.c.mask_words ? q.mask[at + 1] : 0u;
        uint32_t w = (uint32_t)(((u64)w1 << 32 | w0) >> sh);
        const int64_t left = nn - from;
        w = left <= 0 ? 0u : (left >= 32 ? w : w & ((1u << left) - 1));
        if (off < 0) w = w << -off | ((1u << -off) - 1);
        return w;
    };
    // The largest of the tile's scores; far above what the weights are relative
    // to, it takes its place (seldom: m may lag).
    const auto raise = [&](const f32x4 (&s)[2]) __attribute__((always_inline)) {
        float top[2];
        bool far = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
            const auto p16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
            x = fmaxf(__uint_as_float(p16[0]), __uint_as_float(p16[1]));
            const auto p32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
            top[i] = fmaxf(__uint_as_float(p32[0]), __uint_as_float(p32[1])) * a.scale_log2;
            far |= top[i] > m[i] + room(T(), m[i]);
        }
        if (__any(far)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float mm = fmaxf(m[i], top[i] - lift(T(), top[i]));
                l[i] *= factor(m[i], mm);
                m[i] = mm;
            }
        }
    };
    const auto weigh = [&](const f32x4 (&s)[2], int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float base = m[i] == -INFINITY ? 0.0f : m[i];
            s16x4 p;
            float sum = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][x], a.scale_log2, -base));
                sum += e;
                p[x] = (short)T::put(e);
            }
            l[i] += sum;
            *(s16x4*)(weights + buf * S::kRows * S::kWeightRow + (16 * i + col) * S::kWeightRow + 32 * wd + 8 * quad) = p;
            if (quad == 0) max_of(buf, wd, 16 * i + col) = m[i];
        }
    };
    // What the two waves of a row made tile t's weights relative to becomes one,
    // the larger: for this wave's sums and outputs, and the weights as read.
    const auto agree = [&](int buf, s16x8 (&p)[2]) __attribute__((always_inline)) {
        const char* const at = weights + buf * S::kRows * S::kWeightRow + row32 * S::kWeightRow + 16 * half;
        p[0] = *(const s16x8*)at;
        p[1] = *(const s16x8*)(at + 32);
        const float m0 = max_of(buf, 0, row32), m1 = max_of(buf, 1, row32), mm = fmaxf(m0, m1);
        if (__any(mm > m_out || m0 != m1)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float both = fmaxf(max_of(buf, 0, 16 * i + col), max_of(buf, 1, 16 * i + col));
                l[i] *= factor(m[i], both);
                m[i] = both;
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
        }
    };
    const auto products = [&](const char* vt, const s16x8 (&p)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < 2; ++x) o[d] = mfma(T(), value(vt, d, x), p[x], o[d]);
    };
    // The products with the next tile's weights (vector work) between them.
    const auto mix = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
        for (int x = 0; x < 2 * ND; ++x) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
        }
    };

    uint32_t valid[S::kBuffers - 2];                       // keys of the tiles whose copies are in flight, next tile first
    Place place = look_up(0);
#pragma unroll
    for (int i = 0; i < S::kBuffers - 2; ++i) {
        valid[i] = valid_keys(place, i);
        if (i < tiles) issue(place, i);
        place = look_up(i + 1);
    }
    int buf = S::kBuffers - 1;                             // of tile t; t + 1 has the next one
    const auto next = [](int i) __attribute__((always_inline)) { return i + 1 == S::kBuffers ? 0 : i + 1; };
    // tile t's products and tile t + 1's weights
    const auto round = [&](int t, auto is_masked, auto is_started) __attribute__((always_inline)) {
        constexpr bool masked = decltype(is_masked)::value, started = decltype(is_started)::value;
        if (S::kBuffers == 4 && t + 2 < tiles) wait_copies<kCopies>();
        else wait_copies<0>();
        __syncthreads();
        const uint32_t now = valid[0];
        const int b1 = next(buf);
        {
            // the buffer that tile t - 1 has left
            const int ahead = t + S::kBuffers - 1;
#pragma unroll
            for (int i = 0; i + 1 < S::kBuffers - 2; ++i) valid[i] = valid[i + 1];
            valid[S::kBuffers - 3] = valid_keys(place, ahead);
            if (ahead < tiles) issue(place, buf == 0 ? S::kBuffers - 1 : buf - 1);
            place = look_up(ahead + 1);
        }
        f32x4 s[2];
        const bool more = !masked || t + 1 < tiles;
        if (more) scores(lds + b1 * S::kTile, s);
        if constexpr (masked) {
            if (more) {
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
                    const uint32_t see = see_bits(query[i], k0) & now;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int key = 16 * wd + 4 * quad + x;
                        if (!(see >> key & 1)) s[i][x] = -INFINITY;
                        else if (any_odd >> key & 1) s[i][x] = NAN;
                    }
                }
            }
        }
        s16x8 p[2];
        if (started) agree(t & 1, p);
        if (more) raise(s);
        if (started) products(lds + buf * S::kTile, p);
        if (more) weigh(s, (t + 1) & 1);
        if (!masked && started) mix();
        buf = b1;
    };
    int t = -1;
    if (tiles > 0) {
        if (whole > 0 && valid[0] == ~0u) {
            round(t, False(), False());
            for (++t; t + 1 < whole && valid[0] == ~0u; ++t) round(t, False(), True());
        } else {
            round(t, True(), False());
            ++t;
        }
        for (; t < tiles; ++t) round(t, True(), True());
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
