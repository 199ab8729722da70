// ssm_bwd_bf16.hip -- the selective scan's gradient walks for bf16 inputs.
#define GDR_SSM_GRAD_KERNELS
#include "ssm_bwd.h"

namespace gdr {
GDR_INSTANTIATE(__bf16, 64, 64)
GDR_INSTANTIATE(__bf16, 64, 128)
GDR_INSTANTIATE(__bf16, 128, 64)
GDR_INSTANTIATE(__bf16, 128, 128)
}  // namespace gdr
