// Gated feed-forward block on FP8 weights (gfx950): h = act(x Wg + bg) * (x Wu + bu), both products in one pass
// over x on the kernels of linear_tiles.h.
#include "linear_tiles.h"

namespace moe {

hipError_t launch_gated_linear(const LinArgs& args, hipStream_t st) {
    LinArgs a = args;
    a.nt = (int64_t)a.T * a.N * (a.gu ? 3 : 1) >= (32 << 20);
    auto fits = [&](int rows, int cols, int64_t most) { return ceil_div(a.T, rows) * ceil_div(a.N, cols) <= most; };
    if (fits(16, 32, 256)) return run_stream<true, 2, 4, 4>(a, st);
    if (fits(16, 64, 256)) return run_stream<true, 4, 4, 4>(a, st);
    if (fits(64, 64, 256)) return run_deep<true, 1, 4, 4, 1, 4, 2>(a, st);
    if (a.T <= 8) return run_stream<true, 2, 4, 4>(a, st);
    if (fits(64, 128, 256)) return run_deep<true, 2, 4, 2, 2, 4, 1>(a, st);
    if (fits(64, 128, 512) || a.T <= 64) return run_deep<true, 2, 4, 2, 2, 3, 1>(a, st);
    if (fits(128, 256, 256)) {
        if (a.mx) return run_deep_t<kMicro, true, 4, 4, 2, 4, 3, 1>(a, st);
        if (!fits(128, 256, 208) && deep_lds<kBlock, true>(128, 256, 3, a.K / kGroup) <= kLdsBytes)
            return run_deep_t<kBlock, true, 4, 4, 2, 4, 3, 1>(a, st);
        return run_tile_t<kBlock, true, 4, 4, 1, 4>(a, st);
    }
    return a.mx ? run_tile_t<kMicro, true, 8, 4, 1, 4>(a, st) : run_tile_t<kBlock, true, 8, 4, 1, 4>(a, st);
}

}  // namespace moe
