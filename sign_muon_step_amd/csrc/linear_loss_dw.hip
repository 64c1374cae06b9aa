// linear_loss_dw.hip -- the loss's dw_m = g_m^T x_m (linear_loss.hip): both operands' rows
// are k.
#include "loss_tiles.h"

namespace sm {
namespace {

template <int HOW>
void launch_dw(const LossTile &f, hipStream_t s) {
    if constexpr (HOW != kAdd)
        if (f.planes == 1 && !f.out_bf16) {  // parts of tokens
            f.g32 ? launch_wide<kCols32, 1, true, HOW>(f, s) : launch_tiles<kCols16, kCols16, kValues, true, HOW>(f, s);
            return;
        }
    if (!f.g32)
        launch_tiles<kCols16, kCols16, kValues, false, HOW>(f, s);
    else if (f.planes == 3 && f.out_bf16)  // of few tokens: bound by the results
        loss_wide_kernel<kCols32, 128, 128, 3, false, HOW><<<grid_of(f), kWaves * kWave, 0, s>>>(f, tiles_of(f));
    else
        f.planes == 3 ? launch_wide<kCols32, 3, true, HOW>(f, s) : launch_wide<kCols32, 1, false, HOW>(f, s);
}

}  // namespace

void launch_loss_dw(const LossTile &f, hipStream_t s) {
    if (!loss_even(f))
        launch_dw<kUneven>(f, s);
    else
        f.add ? launch_dw<kAdd>(f, s) : launch_dw<kEven>(f, s);
}

}  // namespace sm
