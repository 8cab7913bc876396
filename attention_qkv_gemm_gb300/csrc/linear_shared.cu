// linear_shared.cu -- the linear layer's forward (linear.cu): clusters of lone CTAs that share a tile's sum.
#include "linear_form.cuh"

namespace tfl {

TFL_LINEAR_FORM(shared, 1, kSplit)

}  // namespace tfl
