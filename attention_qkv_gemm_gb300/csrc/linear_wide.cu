// linear_wide.cu -- the linear layer's forward (linear.cu): CTA pairs on tiles as wide as the accumulator.
#include "linear_form.cuh"

namespace tfl {

TFL_LINEAR_FORM(wide, 2, kWide)

}  // namespace tfl
