// rowloss_f16.hip -- the losses over rows of f16 logits.
#include "rowloss_kernels.hpp"

namespace red {
template struct RowLoss<ElemF16>;
} // namespace red
