// mx_act.hip -- the MXFP8 contraction with an epilogue (mx_gemm_kernels.h,
// epilogue.h), one result to a channel.
#define MXQ_ACT_GATED false
#define MXQ_ACT_LAUNCH launch_mx_act
#include "mx_act_launch.h"
