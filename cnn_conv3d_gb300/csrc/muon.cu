// muon.cu -- orthogonalisation of matrices by Newton-Schulz products and the
// momentum step that uses it, with their entry points.
#include <algorithm>
#include <cmath>

#include "cf_internal.h"
#include "cf_ptx.cuh"

namespace cf {
namespace {

constexpr int kNormBlocks = 128;
constexpr float kDown = 0x1p-80f;
constexpr int kTile = 64, kTileK = 16;

__device__ __forceinline__ float load_f(const void* p, int f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
}

// u = g (momentum 0 and m NULL), or the momentum step; partial sums of u^2 and of (kDown u)^2, which
// stands in where the first overflows.
__global__ void __launch_bounds__(256) ns_input_kernel(const void* __restrict__ g, int f32, float* __restrict__ m, float mu,
                                                       int64_t count, int nesterov, float* __restrict__ part) {
    __shared__ float red[8], red2[8];
    float s = 0.f, s2 = 0.f;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < count; i += (int64_t)gridDim.x * blockDim.x) {
        float u = load_f(g, f32, i);
        if (m) {
            const float t = fmaf(mu, m[i], u);
            m[i] = t;
            u = nesterov ? fmaf(mu, t, u) : t;
        }
        s = fmaf(u, u, s);
        u *= kDown;
        s2 = fmaf(u, u, s2);
    }
    for (int o = 16; o; o >>= 1) {
        s += __shfl_down_sync(~0u, s, o);
        s2 += __shfl_down_sync(~0u, s2, o);
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s, red2[threadIdx.x >> 5] = s2;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) s += red[i], s2 += red2[i];
        part[blockIdx.x] = s;
        part[kNormBlocks + blockIdx.x] = s2;
    }
}

// X [k][n] = u / (|u| + eps), transposed where tall.
__global__ void __launch_bounds__(256) ns_scale_kernel(const void* __restrict__ g, int f32, const float* __restrict__ m, float mu,
                                                       int64_t rows, int64_t cols, int nesterov,
                                                       const float* __restrict__ part, float eps, float* __restrict__ X) {
    float s = 0.f, s2 = 0.f;
    for (int i = 0; i < kNormBlocks; ++i) s += part[i], s2 += part[kNormBlocks + i];
    // u / (|u| + eps) as (u pre) inv
    const float pre = isinf(s) ? kDown : 1.f, inv = 1.f / (sqrtf(isinf(s) ? s2 : s) + eps * pre);
    const int64_t count = rows * cols;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < count; i += (int64_t)gridDim.x * blockDim.x) {
        float u = load_f(g, f32, i);
        if (m) u = nesterov ? fmaf(mu, m[i], u) : m[i];
        X[rows > cols ? (i % cols) * rows + i / cols : i] = u * pre * inv;
    }
}

// C [M][N] = al D + be (P [M][K] Q), Q [K][N] or, transposed, [N][K].
__global__ void __launch_bounds__(256) ns_gemm_kernel(const float* __restrict__ P, const float* __restrict__ Q, int q_t,
                                                      const float* __restrict__ D, float al, float be, int64_t M, int64_t N,
                                                      int64_t K, float* __restrict__ C) {
    __shared__ float ps[kTileK][kTile + 1], qs[kTileK][kTile + 1];
    const int64_t i0 = (int64_t)blockIdx.y * kTile, j0 = (int64_t)blockIdx.x * kTile;
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += kTileK) {
        for (int e = threadIdx.x; e < kTile * kTileK; e += 256) {
            const int r = e / kTileK, kk = e % kTileK;
            ps[kk][r] = i0 + r < M && k0 + kk < K ? P[(i0 + r) * K + k0 + kk] : 0.f;
            if (q_t) {
                qs[kk][r] = j0 + r < N && k0 + kk < K ? Q[(j0 + r) * K + k0 + kk] : 0.f;
            } else {
                const int c = e % kTile, kq = e / kTile;
                qs[kq][c] = j0 + c < N && k0 + kq < K ? Q[(k0 + kq) * N + j0 + c] : 0.f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kTileK; ++kk) {
            float p[4], q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = ps[kk][ti + 16 * e], q[e] = qs[kk][tj + 16 * e];
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(p[a], q[b], acc[a][b]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t i = i0 + ti + 16 * a, j = j0 + tj + 16 * b;
            if (i < M && j < N) C[i * N + j] = be * acc[a][b] + (D ? al * D[i * N + j] : 0.f);
        }
}

// o = X, or w = keep w - step X with its bf16 copy; X transposed where tall.
__global__ void __launch_bounds__(256) ns_output_kernel(const float* __restrict__ X, int64_t rows, int64_t cols,
                                                        uint16_t* __restrict__ o, float* __restrict__ w, float keep, float step) {
    const int64_t count = rows * cols;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < count; i += (int64_t)gridDim.x * blockDim.x) {
        float v = X[rows > cols ? (i % cols) * rows + i / cols : i];
        if (w) {
            v = keep * w[i] - step * v;
            w[i] = v;
        }
        if (o) o[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool shape_ok(int64_t rows, int64_t cols) { return rows > 0 && cols > 0; }
bool shape_supported(int64_t rows, int64_t cols) { return rows <= 65536 && cols <= 65536; }

// Workspace of one matrix: norm partials, X twice, A, B.
size_t matrix_bytes(int64_t rows, int64_t cols) {
    const size_t k = (size_t)std::min(rows, cols);
    return 2 * kNormBlocks * sizeof(float) + 256 + ((size_t)rows * cols * 2 + k * k * 2) * sizeof(float);
}

struct Poly {
    int steps;
    float a, b, c, eps;
};
bool poly_ok(const Poly& p) {
    return p.steps >= 1 && std::isfinite(p.a) && std::isfinite(p.b) && std::isfinite(p.c) && p.eps >= 0.f && std::isfinite(p.eps);
}

cf_status run_matrix(const LaunchCtx& ctx, const Poly& p, int64_t rows, int64_t cols, const void* g, int f32, float* m, float mu,
                     int nesterov, uint16_t* o, float* w, float keep, float step, void* ws) {
    const int64_t k = std::min(rows, cols), n = std::max(rows, cols), count = rows * cols;
    float* part = static_cast<float*>(ws);
    float* X = part + 2 * kNormBlocks;
    float* Y = X + (count + 3) / 4 * 4;
    float* A = Y + (count + 3) / 4 * 4;
    float* B = A + (k * k + 3) / 4 * 4;
    const unsigned blocks = (unsigned)std::min<int64_t>((count + 255) / 256, 4 * ctx.num_sms);
    ns_input_kernel<<<kNormBlocks, 256, 0, ctx.stream>>>(g, f32, m, mu, count, nesterov, part);
    ns_scale_kernel<<<blocks, 256, 0, ctx.stream>>>(g, f32, m, mu, rows, cols, nesterov, part, p.eps, X);
    const dim3 kk((unsigned)((k + kTile - 1) / kTile), (unsigned)((k + kTile - 1) / kTile));
    const dim3 kn((unsigned)((n + kTile - 1) / kTile), (unsigned)((k + kTile - 1) / kTile));
    for (int s = 0; s < p.steps; ++s) {
        ns_gemm_kernel<<<kk, 256, 0, ctx.stream>>>(X, X, 1, nullptr, 0.f, 1.f, k, k, n, A);
        ns_gemm_kernel<<<kk, 256, 0, ctx.stream>>>(A, A, 0, A, p.b, p.c, k, k, k, B);
        ns_gemm_kernel<<<kn, 256, 0, ctx.stream>>>(B, X, 0, X, p.a, 1.f, k, n, k, Y);
        std::swap(X, Y);
    }
    ns_output_kernel<<<blocks, 256, 0, ctx.stream>>>(X, rows, cols, o, w, keep, step);
    return cudaGetLastError() == cudaSuccess ? CF_OK : CF_ERR_CUDA;
}

}  // namespace
}  // namespace cf

using namespace cf;

extern "C" {

static cf_status ns_check(const cf_ns_desc* d) {
    if (d == nullptr || d->batch <= 0 || !shape_ok(d->rows, d->cols)) return CF_ERR_INVALID_ARG;
    if (d->dtype != CF_DT_BF16 && d->dtype != CF_DT_F32) return CF_ERR_INVALID_ARG;
    if (!poly_ok(Poly{d->steps, d->a, d->b, d->c, d->eps})) return CF_ERR_INVALID_ARG;
    if (!shape_supported(d->rows, d->cols) || d->batch > (1 << 20) || d->steps > 16) return CF_ERR_UNSUPPORTED;
    return CF_OK;
}

size_t cf_orthogonalize_workspace_size(const cf_ns_desc* desc) {
    return ns_check(desc) == CF_OK ? matrix_bytes(desc->rows, desc->cols) : 0;
}

cf_status cf_orthogonalize(const cf_ns_desc* desc, const void* g, uint16_t* o, void* ws, size_t ws_bytes, void* stream) {
    if (const cf_status st = ns_check(desc); st != CF_OK) return st;
    if (g == nullptr || o == nullptr || !aligned16(g) || !aligned16(o) || !aligned16(ws)) return CF_ERR_INVALID_ARG;
    if (ws == nullptr || ws_bytes < cf_orthogonalize_workspace_size(desc)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    const int f32 = desc->dtype == CF_DT_F32;
    const int64_t count = desc->rows * desc->cols;
    for (int64_t i = 0; i < desc->batch; ++i) {
        const cf_status st = run_matrix(ctx, Poly{desc->steps, desc->a, desc->b, desc->c, desc->eps}, desc->rows, desc->cols,
                                        static_cast<const char*>(g) + i * count * (f32 ? 4 : 2), f32, nullptr, 0.f, 0,
                                        o + i * count, nullptr, 0.f, 0.f, ws);
        if (st != CF_OK) return st;
    }
    return CF_OK;
}

static cf_status muon_check(int32_t count, const cf_muon_param* p) {
    if (count < 0 || (count > 0 && p == nullptr)) return CF_ERR_INVALID_ARG;
    for (int32_t i = 0; i < count; ++i) {
        if (!shape_ok(p[i].rows, p[i].cols) || p[i].w == nullptr || p[i].g == nullptr || p[i].m == nullptr)
            return CF_ERR_INVALID_ARG;
        if (!aligned16(p[i].w) || !aligned16(p[i].w_bf16) || !aligned16(p[i].g) || !aligned16(p[i].m) ||
            !std::isfinite(p[i].scale))
            return CF_ERR_INVALID_ARG;
    }
    for (int32_t i = 0; i < count; ++i)
        if (!shape_supported(p[i].rows, p[i].cols)) return CF_ERR_UNSUPPORTED;
    return CF_OK;
}

size_t cf_muon_workspace_size(int32_t count, const cf_muon_param* params) {
    if (muon_check(count, params) != CF_OK) return 0;
    size_t most = 0;
    for (int32_t i = 0; i < count; ++i) most = std::max(most, matrix_bytes(params[i].rows, params[i].cols));
    return most;
}

cf_status cf_muon_step(int32_t count, const cf_muon_param* params, const cf_muon_hyper* h, void* ws, size_t ws_bytes,
                       void* stream) {
    if (h == nullptr) return CF_ERR_INVALID_ARG;
    const Poly p{h->steps, h->a, h->b, h->c, h->eps};
    if (!poly_ok(p) || !std::isfinite(h->lr) || !std::isfinite(h->momentum) || !std::isfinite(h->weight_decay))
        return CF_ERR_INVALID_ARG;
    if (const cf_status st = muon_check(count, params); st != CF_OK) return st;
    if (!aligned16(ws)) return CF_ERR_INVALID_ARG;
    if (h->steps > 16) return CF_ERR_UNSUPPORTED;
    if (count == 0) return CF_OK;
    if (ws == nullptr || ws_bytes < cf_muon_workspace_size(count, params)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    for (int32_t i = 0; i < count; ++i) {
        const cf_muon_param& q = params[i];
        const cf_status st = run_matrix(ctx, p, q.rows, q.cols, q.g, 1, q.m, h->momentum, h->nesterov != 0, q.w_bf16, q.w,
                                        1.f - h->lr * h->weight_decay, h->lr * q.scale, ws);
        if (st != CF_OK) return st;
    }
    return CF_OK;
}

}  // extern "C"
