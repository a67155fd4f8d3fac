// linear_dgrad.cu -- the product of linear_gemm.cuh for the backward data.
#define CF_LINEAR_OP OP_DGRAD
#include "linear_gemm.cuh"
