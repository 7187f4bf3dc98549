// mx_act_gated.hip -- the MXFP8 contraction with a gated epilogue
// (mx_gemm_kernels.h, epilogue.h): the activation of half of the channels
// times the other half.
#define MXQ_ACT_GATED true
#define MXQ_ACT_LAUNCH launch_mx_act_gated
#include "mx_act_launch.h"
