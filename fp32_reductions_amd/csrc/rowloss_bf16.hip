// rowloss_bf16.hip -- the losses over rows of bf16 logits.
#include "rowloss_kernels.hpp"

namespace red {
template struct RowLoss<ElemBF16>;
} // namespace red
