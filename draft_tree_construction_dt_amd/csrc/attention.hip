// dt_tree_attention: softmax(scale * q k^T) v over a paged cache in one pass
// over the keys, with a running maximum m, sum l and output o per query:
//   m' = max(m, x);  l' = l e^(m - m') + e^(x - m');  o' = o e^(m - m') + e^(x - m') v
//
// Rows.  The G query heads of a key head share its keys, so the matrix rows
// of a request and key head are (chunk row, head in group), G * rows of them;
// a wave takes 32.  A workgroup is WM x WK (x WD) waves: WM x 32 rows, and WK
// groups of waves that take the tiles of KT keys in turn (few rows: the
// waves share the keys out; many rows: they share the tiles).  With heads of
// 256 a wave's sums would not fit its registers: WD = 2 waves then make the
// same scores and half of the outputs each (21 requests' tokens over 1-4 K
// keys: 39 us, with one wave 111).
//
// Products.  Scores are computed transposed, K q^T on 32x32x16 matrix
// instructions, so that a lane holds one query and the tile's keys lie in its
// registers: the softmax needs one exchange (the wave's two halves) a tile.
// The weights then are, as they lie, the right operand of V^T p^T: the sum
// over keys may run in any order, so the left operand is read in the order in
// which the first product left the keys (k = 16 s + 8 j + 4 half + i).
//
// Staging.  K and V tiles go from memory to LDS without passing registers,
// one tile ahead.  16-byte pieces of a row are permuted by the row's number
// on the way (the copy's LDS side is fixed, so the memory side is permuted):
// K by single pieces (a wave reads one piece of 32 rows at once), V by 64-byte
// groups (the transposing read takes 64 bytes of 4 rows at once), which
// spreads both over the 64 banks.
//
// Work.  Each workgroup derives the whole split from the lengths: segments
// (request, key head, row tile) times key units, cut into chunks of equal size
// so that the resident workgroups share the work however ragged the batch is.
// A segment in one chunk is written at once, others by combine_kernel.
//
// Measured (bf16, heads of 128, 4 query heads to a key head, pages of 16): 64
// requests' single tokens over 33-16383 keys, 2.15 GB of cache, in 404 us, 5.3
// TB/s (a copy reads and writes 4.9); two chunks of 2048 over 6-14 K keys in
// 718-775 us, 915-986 TFLOP/s (a large matrix product: 1402), matrix cores 47%
// and vector units 48% busy; one token over 4096 keys in 17 us, all latency
// (behind a page table of 1 M slots the same).
#include "attention_dev.h"

namespace dt {
namespace {

// Row tile by the rows of a key head: up to 32 rows the waves share out the
// keys, up to 64 both, beyond that the rows.  8 requests over 8000 keys, tiles
// of 32 / 64 / 128 rows: 20 rows 64 / 75 / 79 us, 48 rows 79 / 75 / 81, 96 rows
// 113 / 88 / 85.
int tile_rows(const ChunkArgs& c, int G) {
    const int64_t m = (int64_t)c.rows * G;
    return m <= 32 ? 32 : (m <= 64 ? 64 : 128);
}

int slots_for(int mt, int D) {
    if (mt == 32) return kCus * (D == 64 ? 2 : 1);
    return kCus * (D == 256 ? 1 : 2);
}

template <class T, int D>
hipError_t run_rows(const AttentionArgs& a, void* workspace, hipStream_t stream) {
    const int mt = tile_rows(a.c, a.G), slots = slots_for(mt, D);
    using L = Heads<D>;
    if constexpr (D == 256) {
        if (mt == 32) return run<T, L, 1, 2, 2, 32, 1>(a, slots, workspace, stream);
        if (mt == 64) return run<T, L, 2, 1, 2, 64, 1>(a, slots, workspace, stream);
        return run<T, L, 4, 1, 2, 32, 1>(a, slots, workspace, stream);
    } else {
        if (mt == 32) return run<T, L, 1, 4, 1, 32, D == 64 ? 2 : 1>(a, slots, workspace, stream);
        if (mt == 64) return run<T, L, 2, 2, 1, 32, 2>(a, slots, workspace, stream);
        return run<T, L, 4, 1, 1, 64, 2>(a, slots, workspace, stream);
    }
}

template <class T>
hipError_t run_type(const AttentionArgs& a, void* workspace, hipStream_t stream) {
    switch (a.kv.D) {
    case 64: return run_rows<T, 64>(a, workspace, stream);
    case 128: return run_rows<T, 128>(a, workspace, stream);
    default: return run_rows<T, 256>(a, workspace, stream);
    }
}

}  // namespace

size_t attention_workspace(const ChunkArgs& c, int Hkv, int Hq, int D) {
    const int G = Hq / Hkv, mt = tile_rows(c, G), slots = slots_for(mt, D);
    const int64_t segments = (int64_t)c.B * Hkv * (((int64_t)c.rows * G + mt - 1) / mt);
    return partial_bytes(segments, slots, mt, D);
}

hipError_t launch_attention(const AttentionArgs& a, int dtype, void* workspace, hipStream_t stream) {
    return dtype == DT_DTYPE_BF16 ? run_type<Bf16>(a, workspace, stream)
                                  : run_type<F16>(a, workspace, stream);
}

}  // namespace dt
