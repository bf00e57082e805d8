// rowloss_f32.hip -- the losses over rows of f32 logits.
#include "rowloss_kernels.hpp"

namespace red {
template struct RowLoss<ElemF32>;
} // namespace red
