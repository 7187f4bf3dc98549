// i8_act.hip -- the product of 8-bit codes with an epilogue (i8_kernels.h,
// epilogue.h), one result to a channel: bias, activation, residual.
#define MXQ_ACT_GATED false
#define MXQ_ACT_GEMM launch_i8_gemm_act
#define MXQ_ACT_LINEAR launch_i8_linear_fused_act
#include "i8_act_launch.h"
