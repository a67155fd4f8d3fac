// linear_wgrad.cu -- the product of linear_gemm.cuh for the backward weight.
#define CF_LINEAR_OP OP_WGRAD
#include "linear_gemm.cuh"
