// Gated feed-forward block on FP8 weights (gfx950): h = act(x Wg + bg) * (x Wu + bu), both products in one pass
// over x on the kernels of linear_tiles.h, whose waves hold the gate and the up sums of the same columns: the
// product needs no exchange and no second read of x.  Bound by the weight stream for few rows (1 x 7168 x 2048:
// 8.5-9.0 us, 29 MB), by the matrix cores for many (4096 x 7168 x 2048: 91-97 us, 2.5-2.6 PFLOP/s), by
// latency between (2047 x 768 x 1152: 10.5 us, with the sums kept 13.1).
#include "linear_tiles.h"

namespace moe {

// Variant by the number of workgroups that a tile size makes (256: one per CU), columns counted as w's, two for
// each of h.  As for the linear layer, but that 64 x 64 tiles follow on the stream kernel with 32 columns (48 x 4096 x
// 1536: 9.4 us, the stream kernel with 64 columns 11.4; 64 x 768 x 1152: 4.9 and 5.3; with 32 14.2 and 5.5).
//   * Stream kernel: 32 x 2816 x 768 6.3 us, 64 x 64 tiles 7.4; up to eight rows always (1 x 2816 x 8192: 10.0, 10.3).
//   * Deep 64 x 64 tiles: 128 x 4096 x 2048 10.1, 64 x 128 tiles 14.9.
//   * Deep 64 x 128 tiles, four stages: 512 x 4096 x 2048 16.0, three stages 20.7, 64 x 64 tiles 19.1; three:
//     1024 x 4096 x 2048 23.4, four 29.6, 128 x 256 tiles 28.2.
//   * 128 x 256 tiles with eight waves (2048 x 4096 x 2048: 34.9, k_linear_tile 35.1), or 64 x 256 k_linear_tile
//     where they leave more than a few CUs idle (2047 x 768 x 1152: 10.6, 10.9); beyond, k_linear_tile on 128 x 256 with two
//     workgroups per CU (4096 x 7168 x 2048: 93-97, 108 with the others).
hipError_t launch_gated_linear(const LinArgs& args, hipStream_t st) {
    LinArgs a = args;
    a.nt = (int64_t)a.T * a.N * (a.gu ? 3 : 1) >= (32 << 20);   // bytes written: past the caches, as the linear layer's
    auto fits = [&](int rows, int cols, int64_t most) { return ceil_div(a.T, rows) * ceil_div(a.N, cols) <= most; };
    if (fits(16, 32, 256)) return run_stream<true, 2, 4, 4>(a, st);
    if (fits(64, 64, 256)) return run_deep<true, 1, 4, 4, 1, 4, 2>(a, st);
    if (a.T <= 8) return run_stream<true, 2, 4, 4>(a, st);
    if (fits(64, 128, 256)) return run_deep<true, 2, 4, 2, 2, 4, 1>(a, st);
    if (fits(64, 128, 512) || a.T <= 64) return run_deep<true, 2, 4, 2, 2, 3, 1>(a, st);
    if (fits(128, 256, 256)) {
        static_assert(deep_lds<kMicro, true>(128, 256, 3, 1) <= kLdsBytes, "for every K: the scales are in the stages");
        if (a.mx) return run_deep_t<kMicro, true, 4, 4, 2, 4, 3, 1>(a, st);
        if (!fits(128, 256, 208) && deep_lds<kBlock, true>(128, 256, 3, a.K / kGroup) <= kLdsBytes)
            return run_deep_t<kBlock, true, 4, 4, 2, 4, 3, 1>(a, st);
        return run_tile_t<kBlock, true, 4, 4, 1, 4>(a, st);
    }
    return a.mx ? run_tile_t<kMicro, true, 8, 4, 1, 4>(a, st) : run_tile_t<kBlock, true, 8, 4, 1, 4>(a, st);
}

}  // namespace moe
