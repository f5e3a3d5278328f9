// FP8 matrix product with bias, activation and residual in its epilogue (gfx950):
//   y = act(dequant(x) @ dequant(w) + bias) + residual,
// on the kernels of linear_tiles.h.
#include "linear_tiles.h"

namespace moe {

// Variant by the number of workgroups that a tile size makes (256: one per CU), times measured with a
// residual.
//   * The stream kernel while its 16-row tiles are no more than that: the narrower of its two (32 x 4096 x 512:
//     6.7 us on 16 columns, 11.7 on 32), then the other (48 x 7168 x 2048: 10.0; deep 64 x 64 tiles 13.2).  More
//     tiles would read the activations again and again (32 x 2048 x 5632: 8.7, deep 6.7).
//   * Deep 64 x 64 tiles with two sets of waves, which halve a tile's chain of K blocks (64 x 7168 x 7168: 14.1 us,
//     one set 16.7, stream tiles 20; 128 x 4096 x 4096: 9.6, deep 64 x 128 tiles 15).
//   * Up to eight rows, whose re-reading costs little, the stream kernel again where those would be more tiles
//     (1 x 7168 x 18432: 24 us, 64 x 128 tiles 30; 16 x 2048 x 20480: 13.7 and 10.3).
//   * Deep 64 x 128 tiles, with four stages where each has a CU to itself (512 x 4096 x 4096: 15.6 us, a second set
//     of waves 17.6, k_linear_tile on the same tiles 22.2; 192 x 7168 x 7168: 22.8) and three, which fit twice,
//     while two share one (1024 x 4096 x 4096: 23.2, four stages 29.0) or there is one row of tiles
//     (64 x 4096 x 131072: 95, 128 x 256 tiles 103).
//   * Then 128 x 256 tiles.  While each has a CU to itself, deep copies with eight waves (2048 x 4096 x 4096:
//     36.7 us, MXFP8 43.9; k_linear_tile on 64 x 256 tiles 37.9 and 50.7, deep 64 x 128 tiles 44.6 and 48.9),
//     but with 128-element scales 64 x 256 k_linear_tile if they leave more than a few CUs idle (1300 x 2048 x
//     4096, 176 tiles: 18.7 and 19.2; MXFP8 23.1 and 22.5), or from K = 15232 on, where the scales of all K
//     blocks do not fit beside the stages.
//   * k_linear_tile beyond, two workgroups per CU (4096 x 4096 x 4096: 63 us; deep 78, 64 x 256 tiles 77).
hipError_t launch_linear(const LinArgs& args, hipStream_t st) {
    LinArgs a = args;
    // Outputs larger than the L2s together leave past them: they would evict the operands that the
    // running tiles share (16384 x 4096 x 4096 in bf16: 238 -> 224 us).
    a.nt = (int64_t)a.T * a.N * (a.out_bf16 ? 2 : 4) >= (32 << 20);
    auto fits = [&](int rows, int cols, int64_t most) { return ceil_div(a.T, rows) * ceil_div(a.N, cols) <= most; };
    if (fits(16, 16, 256)) return run_stream<false, 1, 4, 4>(a, st);
    if (fits(16, 32, 256)) return run_stream<false, 2, 4, 4>(a, st);
    if (fits(64, 64, 256)) return run_deep<false, 1, 4, 4, 1, 4, 2>(a, st);
    if (a.T <= 8) return run_stream<false, 2, 4, 4>(a, st);
    if (fits(64, 128, 256)) return run_deep<false, 2, 4, 2, 2, 4, 1>(a, st);
    if (fits(64, 128, 512) || a.T <= 64) return run_deep<false, 2, 4, 2, 2, 3, 1>(a, st);
    if (fits(128, 256, 256)) {
        static_assert(deep_lds<kMicro, false>(128, 256, 3, 1) <= kLdsBytes, "for every K: the scales are in the stages");
        if (a.mx) return run_deep_t<kMicro, false, 4, 4, 2, 4, 3, 1>(a, st);
        if (!fits(128, 256, 208) && deep_lds<kBlock, false>(128, 256, 3, a.K / kGroup) <= kLdsBytes)
            return run_deep_t<kBlock, false, 4, 4, 2, 4, 3, 1>(a, st);
        return run_tile_t<kBlock, false, 4, 4, 1, 4>(a, st);
    }
    return a.mx ? run_tile_t<kMicro, false, 8, 4, 1, 4>(a, st) : run_tile_t<kBlock, false, 8, 4, 1, 4>(a, st);
}

}  // namespace moe
