// linear_loss_walk.cpp, and besides it the states that the pass over rows'
// factors reads (fp16 rows with factors of their own).
#include "linear_loss.h"

#define launch_coef factors_alone
#include "linear_loss_walk.cpp"
#undef launch_coef

namespace tgemm {
namespace loss {

hipError_t launch_coef(const CoefArgs &a, hipStream_t stream)
{
    if (a.half && a.grad_step != 0) {
        if (a.D < 1 || a.ldx < a.D) fail("states without a width", 0, 0);
        rows(a.X, a.T, a.D, a.ldx, 2, false, "states");
        loads += a.T;
    }
    return factors_alone(a, stream);
}

}  // namespace loss
}  // namespace tgemm
