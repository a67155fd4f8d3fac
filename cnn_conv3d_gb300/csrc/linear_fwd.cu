// linear_fwd.cu -- the product of linear_gemm.cuh for the forward.
#define CF_LINEAR_OP OP_FWD
#include "linear_gemm.cuh"
