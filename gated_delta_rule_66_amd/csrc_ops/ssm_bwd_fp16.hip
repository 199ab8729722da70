// ssm_bwd_fp16.hip -- the selective scan's gradient walks for fp16 inputs.
#define GDR_SSM_GRAD_KERNELS
#include "ssm_bwd.h"

namespace gdr {
GDR_INSTANTIATE(_Float16, 64, 64)
GDR_INSTANTIATE(_Float16, 64, 128)
GDR_INSTANTIATE(_Float16, 128, 64)
GDR_INSTANTIATE(_Float16, 128, 128)
}  // namespace gdr
