// i8_act_gated.hip -- the product of 8-bit codes with a gated epilogue
// (i8_kernels.h, epilogue.h): the activation of half of the channels times the
// other half.
#define MXQ_ACT_GATED true
#define MXQ_ACT_GEMM launch_i8_gemm_act_gated
#define MXQ_ACT_LINEAR launch_i8_linear_fused_act_gated
#include "i8_act_launch.h"
