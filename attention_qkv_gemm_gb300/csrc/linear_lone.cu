// linear_lone.cu -- the linear layer's forward (linear.cu): lone CTAs.
#include "linear_form.cuh"

namespace tfl {

TFL_LINEAR_FORM(lone, 1, kNarrow)

}  // namespace tfl
