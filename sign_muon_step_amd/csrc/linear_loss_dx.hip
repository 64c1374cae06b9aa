// linear_loss_dx.hip -- the loss's dx = g w (linear_loss.hip): w's rows are k, and g's
// rows run along k.
#include "loss_tiles.h"

namespace sm {
namespace {

template <int HOW>
void launch_dx(const LossTile &f, hipStream_t s) {
    if (!f.g32)
        f.out_bf16 ? launch_tiles<kRows16, kCols16, kValues, false, HOW>(f, s)
                   : launch_tiles<kRows16, kCols16, kValues, true, HOW>(f, s);
    else if (f.planes == 3)
        launch_wide<kRows32, 3, true, HOW>(f, s);
    else
        f.out_bf16 ? launch_wide<kRows32, 1, false, HOW>(f, s) : launch_wide<kRows32, 1, true, HOW>(f, s);
}

}  // namespace

void launch_loss_dx(const LossTile &f, hipStream_t s) {
    loss_even(f) ? launch_dx<kEven>(f, s) : launch_dx<kUneven>(f, s);
}

}  // namespace sm
