// linear_pair.cu -- the linear layer's forward (linear.cu): CTA pairs on narrower tiles.
#include "linear_form.cuh"

namespace tfl {

TFL_LINEAR_FORM(pair, 2, kNarrow)

}  // namespace tfl
