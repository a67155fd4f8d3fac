// linear.cu -- matrix products of bf16 rows with bias, activation and residual in the epilogue (forward), with the activation's
// derivative in it (backward data), and summed over the rows (backward weight), with their entry points.
#include <algorithm>
#include <cmath>

#include "cf_internal.h"
#include "cf_ptx.cuh"

namespace cf {
namespace {

enum { ACT_LRELU = CF_ACT_LRELU, ACT_SILU = CF_ACT_SILU, ACT_GELU = CF_ACT_GELU };

constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 1 / (1 + exp(-t))
__device__ __forceinline__ float sigmoid(float t) { return __fdividef(1.f, 1.f + __expf(-t)); }

__device__ __forceinline__ float act_of(int act, float slope, float z) {
    if (act == ACT_LRELU) return z > 0.f ? z : slope * z;
    return z * sigmoid(act == ACT_SILU ? z : kGeluA * fmaf(kGeluB * z, z * z, z));
}
__device__ __forceinline__ float act_grad(int act, float slope, float z) {
    if (act == ACT_LRELU) return z > 0.f ? 1.f : slope;
    z = z > 100.f ? 100.f : z < -100.f ? -100.f : z;  // 1 and 0 beyond, where products with 1 - e would be inf times 0
    if (act == ACT_SILU) {
        const float e = sigmoid(z);
        return fmaf(z * e, 1.f - e, e);
    }
    const float e = sigmoid(kGeluA * fmaf(kGeluB * z, z * z, z));
    return fmaf(z * e * (1.f - e), kGeluA * fmaf(3.f * kGeluB * z, z, 1.f), e);
}

// What the epilogue of a product needs: D [m][n], pitch values a row.
struct Epi {
    const float* bias;
    const void* add;        // residual
    const uint16_t* pre_in; // backward data: the derivative's argument
    uint16_t* pre_out;
    void* out;
    int64_t pitch;
    int act, f32, accumulate;
    float slope, scale;
};

enum { OP_FWD = CF_LINEAR_FWD, OP_DGRAD = CF_LINEAR_DGRAD, OP_WGRAD = CF_LINEAR_WGRAD };

template <int OP>
__device__ __forceinline__ void finish(const Epi& E, int64_t i, int j, float acc) {
    const int64_t o = i * E.pitch + j;
    float v;
    if (OP == OP_FWD) {
        const float z = acc + (E.bias ? E.bias[j] : 0.f);
        if (E.pre_out) E.pre_out[o] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
        v = E.scale * act_of(E.act, E.slope, z);
    } else {
        v = E.scale * acc;
        if (OP == OP_DGRAD && E.pre_in) v *= act_grad(E.act, E.slope, bf16_bits_to_float(E.pre_in[o]));
    }
    if (OP == OP_WGRAD) {
        float* d = static_cast<float*>(E.out) + o;
        *d = E.accumulate ? *d + v : v;
        return;
    }
    if (E.f32) {
        if (E.add) v += static_cast<const float*>(E.add)[o];
        static_cast<float*>(E.out)[o] = v;
    } else {
        if (E.add) v += bf16_bits_to_float(static_cast<const uint16_t*>(E.add)[o]);
        static_cast<uint16_t*>(E.out)[o] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

// A(i, k) and B(j, k) at their strides.
struct Operands {
    const uint16_t *a, *b;
    int64_t ai, ak, bj, bk, m, k;
    int n;
};

// 64 x 64 outputs to a block, 4 x 4 to a thread, 16 of the contracted axis at a time.
template <int OP>
__global__ void __launch_bounds__(256) linear_kernel(const Operands P, const Epi E) {
    __shared__ float as[16][65], bs[16][65];
    const int64_t i0 = (int64_t)blockIdx.x * 64;
    const int j0 = blockIdx.y * 64, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < P.k; k0 += 16) {
        for (int e = threadIdx.x; e < 1024; e += 256) {
            // along the axis that is contiguous
            const int ka = P.ak == 1 ? e & 15 : e >> 6, ia = P.ak == 1 ? e >> 4 : e & 63;
            const int kb = P.bk == 1 ? e & 15 : e >> 6, jb = P.bk == 1 ? e >> 4 : e & 63;
            as[ka][ia] = i0 + ia < P.m && k0 + ka < P.k ? bf16_bits_to_float(P.a[(i0 + ia) * P.ai + (k0 + ka) * P.ak]) : 0.f;
            bs[kb][jb] = j0 + jb < P.n && k0 + kb < P.k ? bf16_bits_to_float(P.b[(j0 + jb) * P.bj + (k0 + kb) * P.bk]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(as[k][ty + 16 * a], bs[k][tx + 16 * b], acc[a][b]);
        __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (i0 + ty + 16 * a < P.m && j0 + tx + 16 * b < P.n) finish<OP>(E, i0 + ty + 16 * a, j0 + tx + 16 * b, acc[a][b]);
}

// db = scale sum of the rows of dz: 32 columns to a block.
__global__ void __launch_bounds__(256) linear_bias_kernel(const uint16_t* dz, int64_t rows, int n, int64_t pitch, float scale, int accumulate,
                                                          float* db) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (j < n)
        for (int64_t i = q; i < rows; i += 8) s += bf16_bits_to_float(dz[i * pitch + j]);
    red[q][lane] = s;
    __syncthreads();
    if (q == 0 && j < n) {
        for (int i = 1; i < 8; ++i) s += red[i][lane];
        db[j] = accumulate ? db[j] + scale * s : scale * s;
    }
}

__global__ void __launch_bounds__(256) linear_act_bwd_kernel(const void* dy, int f32, const uint16_t* pre, uint16_t* dz, int64_t rows, int n,
                                                             int64_t pitch, int act, float slope, float scale) {
    for (int64_t e = blockIdx.x * (int64_t)256 + threadIdx.x; e < rows * n; e += (int64_t)gridDim.x * 256) {
        const int64_t i = e / n, o = i * pitch + (e - i * n);
        const float d = f32 ? static_cast<const float*>(dy)[o] : bf16_bits_to_float(static_cast<const uint16_t*>(dy)[o]);
        dz[o] = __bfloat16_as_ushort(__float2bfloat16_rn(scale * d * act_grad(act, slope, bf16_bits_to_float(pre[o]))));
    }
}

// --------------------------------------------------------------------------------------------------------------------------- host
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
cf_status status_of() { return cudaGetLastError() == cudaSuccess ? CF_OK : CF_ERR_CUDA; }

cf_status check(const cf_linear_desc* d) {
    if (d == nullptr || d->rows < 0 || d->k <= 0 || d->n <= 0) return CF_ERR_INVALID_ARG;
    if (d->act < CF_ACT_LRELU || d->act > CF_ACT_GELU || !std::isfinite(d->slope) || !std::isfinite(d->scale)) return CF_ERR_INVALID_ARG;
    if (d->dtype != CF_DT_BF16 && d->dtype != CF_DT_F32) return CF_ERR_INVALID_ARG;
    if ((d->x_pitch && d->x_pitch < d->k) || (d->y_pitch && d->y_pitch < d->n)) return CF_ERR_INVALID_ARG;
    if (d->rows >= (int64_t)1 << 31 || d->k > 1 << 20 || d->n > 1 << 20 || d->x_pitch >= 1 << 28 || d->y_pitch >= 1 << 28)
        return CF_ERR_UNSUPPORTED;
    return CF_OK;
}
int64_t x_pitch(const cf_linear_desc* d) { return d->x_pitch ? d->x_pitch : d->k; }
int64_t y_pitch(const cf_linear_desc* d) { return d->y_pitch ? d->y_pitch : d->n; }

template <int OP>
cf_status product(const LaunchCtx& ctx, const Operands& P, const Epi& E) {
    linear_kernel<OP><<<dim3((unsigned)((P.m + 63) / 64), (unsigned)((P.n + 63) / 64)), 256, 0, ctx.stream>>>(P, E);
    return status_of();
}

}  // namespace
}  // namespace cf

using namespace cf;

extern "C" {

size_t cf_linear_workspace_size(const cf_linear_desc* desc, int32_t op) {
    if (check(desc) != CF_OK || op < CF_LINEAR_FWD || op > CF_LINEAR_WGRAD) return 0;
    return 0;
}

cf_status cf_linear_fwd(const cf_linear_desc* desc, const uint16_t* x, const uint16_t* w, const float* bias, const void* residual, void* y,
                        uint16_t* pre, void* ws, size_t ws_bytes, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    if (desc->rows == 0) return CF_OK;
    if (!x || !w || !y) return CF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)x, (const void*)w, (const void*)bias, residual, (const void*)y, (const void*)pre, (const void*)ws})
        if (!aligned16(p)) return CF_ERR_INVALID_ARG;
    if (ws_bytes < cf_linear_workspace_size(desc, CF_LINEAR_FWD)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    const Operands P{x, w, x_pitch(desc), 1, desc->k, 1, desc->rows, desc->k, desc->n};
    return product<OP_FWD>(ctx, P, Epi{bias, residual, nullptr, pre, y, y_pitch(desc), desc->act, desc->dtype == CF_DT_F32, 0, desc->slope, desc->scale});
}

cf_status cf_linear_act_bwd(const cf_linear_desc* desc, const void* dy, const uint16_t* pre, uint16_t* dz, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    if (desc->rows == 0) return CF_OK;
    if (!dy || !pre || !dz || !aligned16(dy) || !aligned16(pre) || !aligned16(dz)) return CF_ERR_INVALID_ARG;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    const int64_t blocks = std::min<int64_t>((desc->rows * desc->n + 255) / 256, 8 * ctx.num_sms);
    linear_act_bwd_kernel<<<(unsigned)blocks, 256, 0, ctx.stream>>>(dy, desc->dtype == CF_DT_F32, pre, dz, desc->rows, desc->n, y_pitch(desc),
                                                                    desc->act, desc->slope, desc->scale);
    return status_of();
}

cf_status cf_linear_dgrad(const cf_linear_desc* desc, const uint16_t* dz, const uint16_t* w, const uint16_t* pre, const void* add, void* dx,
                          void* ws, size_t ws_bytes, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    if (desc->rows == 0) return CF_OK;
    if (!dz || !w || !dx) return CF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)dz, (const void*)w, (const void*)pre, add, (const void*)dx, (const void*)ws})
        if (!aligned16(p)) return CF_ERR_INVALID_ARG;
    if (ws_bytes < cf_linear_workspace_size(desc, CF_LINEAR_DGRAD)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    const Operands P{dz, w, y_pitch(desc), 1, 1, desc->k, desc->rows, desc->n, desc->k};
    return product<OP_DGRAD>(ctx, P, Epi{nullptr, add, pre, nullptr, dx, x_pitch(desc), desc->act, desc->dtype == CF_DT_F32, 0, desc->slope, desc->scale});
}

cf_status cf_linear_wgrad(const cf_linear_desc* desc, const uint16_t* x, const uint16_t* dz, float* dw, float* db, int32_t accumulate, void* ws,
                          size_t ws_bytes, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    if ((desc->rows && (!x || !dz)) || !dw) return CF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)x, (const void*)dz, (const void*)dw, (const void*)db, (const void*)ws})
        if (!aligned16(p)) return CF_ERR_INVALID_ARG;
    if (ws_bytes < cf_linear_workspace_size(desc, CF_LINEAR_WGRAD)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    const Operands P{dz, x, 1, y_pitch(desc), 1, x_pitch(desc), desc->n, desc->rows, desc->k};
    if (db) {
        linear_bias_kernel<<<(desc->n + 31) / 32, 256, 0, ctx.stream>>>(dz, desc->rows, desc->n, y_pitch(desc), desc->scale, accumulate, db);
        if (const cf_status st = status_of(); st != CF_OK) return st;
    }
    return product<OP_WGRAD>(ctx, P, Epi{nullptr, nullptr, nullptr, nullptr, dw, desc->k, CF_ACT_LRELU, 1, accumulate, 1.f, desc->scale});
}

}  // extern "C"
