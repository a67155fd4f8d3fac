// group_norm.cu -- group normalisation of NDHWC volumes with the block's
// activation and pooling, forward and backward, and their entry points.
//
// Forward and backward each are: per-chunk channel sums, their reduction to
// what a group needs, and one pass that writes the output.
#include <algorithm>

#include "cf_internal.h"
#include "cf_ptx.cuh"

namespace cf {
namespace {

constexpr int kThreads = 256;

struct GnArgs {
    int64_t n, d, h, w, s;  // s = d*h*w
    int c, groups, cg;
    int64_t xp, yp;
    float slope, eps;
    int chunks;      // chunks of rows a sample is cut into
    int64_t rows;    // rows (voxels, or pooled windows) of a chunk
    int64_t total;   // rows of a sample
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<uint16_t>(uint16_t v) { return bf16_bits_to_float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f<uint16_t>(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float (&f)[V]) {
    const Pack<T, V> t = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = to_f<T>(t.v[e]);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&f)[V]) {
    Pack<T, V> t;
#pragma unroll
    for (int e = 0; e < V; ++e) t.v[e] = from_f<T>(f[e]);
    *reinterpret_cast<Pack<T, V>*>(p) = t;
}

template <int ACT>
__device__ __forceinline__ float act_of(float u, float slope) {
    if (ACT == CF_ACT_SILU) return u / (1.f + expf(-u));
    return u > 0.f ? u : slope * u;
}
template <int ACT>
__device__ __forceinline__ float act_grad(float u, float slope) {
    if (ACT == CF_ACT_SILU) {
        const float e = 1.f / (1.f + expf(-u));
        return e * (1.f + u * (1.f - e));
    }
    return u > 0.f ? 1.f : slope;
}

// The x offset (in values) of voxel k of row r of a sample: a voxel, or voxel k of a pooled window.
template <int POOL>
__device__ __forceinline__ int64_t voxel_of(const GnArgs& A, int64_t n, int64_t r, int k) {
    if (POOL == CF_POOL_NONE) return (n * A.s + r) * A.xp;
    const int64_t w2 = A.w / 2, h2 = A.h / 2;
    const int64_t pw = r % w2, q = r / w2, ph = q % h2, pd = q / h2;
    return (n * A.s + ((2 * pd + (k >> 2)) * A.h + 2 * ph + ((k >> 1) & 1)) * A.w + 2 * pw + (k & 1)) * A.xp;
}

// Channel means and sums of squared deviations of one chunk (part[n][chunk][c] float2).
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_stats_kernel(GnArgs A, const T* __restrict__ x, float2* __restrict__ part) {
    __shared__ float sm[kThreads * V], sq[kThreads * V];
    const int cols = min(A.c / V - (int)blockIdx.y * kThreads, kThreads), lanes = kThreads / cols;
    const int col = threadIdx.x % cols, lane = threadIdx.x / cols;
    const int64_t n = blockIdx.z, r0 = blockIdx.x * A.rows, r1 = min(r0 + A.rows, A.total);
    const int c0 = ((int)blockIdx.y * kThreads + col) * V;
    float k[V], s[V], q[V];
    int64_t cnt = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) k[e] = s[e] = q[e] = 0.f;
    if (lane < lanes)
        for (int64_t r = r0 + lane; r < r1; r += lanes) {
            float f[V];
            load<T, V>(x + (n * A.s + r) * A.xp + c0, f);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (cnt == 0) k[e] = f[e];
                const float t = f[e] - k[e];
                s[e] += t;
                q[e] = fmaf(t, t, q[e]);
            }
            ++cnt;
        }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float m = cnt ? s[e] / (float)cnt : 0.f;
        sm[threadIdx.x * V + e] = k[e] + m;
        sq[threadIdx.x * V + e] = fmaxf(q[e] - s[e] * m, 0.f);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < cols * V; i += kThreads) {
        const int cc = i / V, e = i % V;
        float mean = 0.f, m2 = 0.f, have = 0.f;
        for (int l = 0; l < lanes; ++l) {
            const int64_t left = r1 - r0 - l;
            const float nb = left > 0 ? (float)((left + lanes - 1) / lanes) : 0.f;
            if (nb == 0.f) break;
            const float mb = sm[(l * cols + cc) * V + e], qb = sq[(l * cols + cc) * V + e];
            const float tot = have + nb, d = mb - mean;
            mean += d * (nb / tot);
            m2 += qb + d * d * (have * nb / tot);
            have = tot;
        }
        part[(n * A.chunks + blockIdx.x) * A.c + (int)blockIdx.y * kThreads * V + i] = make_float2(mean, m2);
    }
}

__device__ __forceinline__ double block_sum(double v, double* red) {
    for (int o = 16; o; o >>= 1) v += __shfl_down_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) t += red[i];
    __syncthreads();
    return t;
}

// mean and rstd of a group from the chunks' channel statistics.
__global__ void __launch_bounds__(kThreads) gn_stats_reduce_kernel(GnArgs A, const float2* __restrict__ part,
                                                                  float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ double red[kThreads / 32];
    const int64_t n = blockIdx.x / A.groups;
    const int g = blockIdx.x % A.groups;
    const int items = A.chunks * A.cg;
    const double count = (double)A.s * A.cg;
    double sum = 0.0;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int ch = i / A.cg;
        const double nb = (double)min(A.rows, A.total - ch * A.rows);
        sum += nb * (double)part[(n * A.chunks + ch) * A.c + g * A.cg + i % A.cg].x;
    }
    const double mu = block_sum(sum, red) / count;
    double m2 = 0.0;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int ch = i / A.cg;
        const double nb = (double)min(A.rows, A.total - ch * A.rows);
        const float2 p = part[(n * A.chunks + ch) * A.c + g * A.cg + i % A.cg];
        m2 += (double)p.y + nb * ((double)p.x - mu) * ((double)p.x - mu);
    }
    const double var = block_sum(m2, red) / count;
    if (threadIdx.x == 0) {
        mean[blockIdx.x] = (float)mu;
        rstd[blockIdx.x] = (float)(1.0 / sqrt(var + (double)A.eps));
    }
}

// u = a (x - mean) + b: taking the mean off first keeps u exact to its own size where |mean| is large against the deviation.
template <int V>
__device__ __forceinline__ void affine(const GnArgs& A, int64_t n, int c0, const float* __restrict__ gamma,
                                       const float* __restrict__ beta, const float* __restrict__ mean,
                                       const float* __restrict__ rstd, float (&a)[V], float (&b)[V], float (&m)[V],
                                       float (&r)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int g = (c0 + e) / A.cg;
        m[e] = mean[n * A.groups + g];
        r[e] = rstd[n * A.groups + g];
        a[e] = (gamma ? gamma[c0 + e] : 1.f) * r[e];
        b[e] = beta ? beta[c0 + e] : 0.f;
    }
}

template <typename T, int V, int POOL, int ACT>
__global__ void __launch_bounds__(kThreads) gn_apply_kernel(GnArgs A, const T* __restrict__ x, const float* __restrict__ gamma,
                                                           const float* __restrict__ beta, const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, T* __restrict__ y) {
    const int cols = min(A.c / V - (int)blockIdx.y * kThreads, kThreads), lanes = kThreads / cols;
    const int col = threadIdx.x % cols, lane = threadIdx.x / cols;
    if (lane >= lanes) return;
    const int64_t n = blockIdx.z, r0 = blockIdx.x * A.rows, r1 = min(r0 + A.rows, A.total);
    const int c0 = ((int)blockIdx.y * kThreads + col) * V;
    float a[V], b[V], m[V], rs[V];
    affine<V>(A, n, c0, gamma, beta, mean, rstd, a, b, m, rs);
    for (int64_t r = r0 + lane; r < r1; r += lanes) {
        float o[V], f[V];
#pragma unroll
        for (int k = 0; k < (POOL == CF_POOL_NONE ? 1 : 8); ++k) {
            load<T, V>(x + voxel_of<POOL>(A, n, r, k) + c0, f);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float u = fmaf(a[e], f[e] - m[e], b[e]);
                if (POOL == CF_POOL_MAX)
                    o[e] = k == 0 || u > o[e] ? u : o[e];
                else if (POOL == CF_POOL_AVG)
                    o[e] = (k == 0 ? 0.f : o[e]) + act_of<ACT>(u, A.slope);
                else
                    o[e] = u;
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = POOL == CF_POOL_AVG ? 0.125f * o[e] : act_of<ACT>(o[e], A.slope);
        store<T, V>(y + (n * A.total + r) * A.yp + c0, o);
    }
}

// du of the rows' voxels; PASS 0: channel sums of du and du xh of a chunk (part[n][chunk][c] float2);
// PASS 1: dx from the groups' means s1, s2 (coef[n][groups] float2).
template <typename T, int V, int POOL, int ACT, int PASS>
__global__ void __launch_bounds__(kThreads) gn_bwd_kernel(GnArgs A, const T* __restrict__ x, const float* __restrict__ gamma,
                                                         const float* __restrict__ beta, const float* __restrict__ mean,
                                                         const float* __restrict__ rstd, const T* __restrict__ dy,
                                                         const float2* __restrict__ coef, float2* __restrict__ part,
                                                         T* __restrict__ dx) {
    __shared__ float sb[PASS == 0 ? kThreads * V : 1], sg[PASS == 0 ? kThreads * V : 1];
    const int cols = min(A.c / V - (int)blockIdx.y * kThreads, kThreads), lanes = kThreads / cols;
    const int col = threadIdx.x % cols, lane = threadIdx.x / cols;
    const int64_t n = blockIdx.z, r0 = blockIdx.x * A.rows, r1 = min(r0 + A.rows, A.total);
    const int c0 = ((int)blockIdx.y * kThreads + col) * V;
    constexpr int K = POOL == CF_POOL_NONE ? 1 : 8;
    float db[V], dg[V];
#pragma unroll
    for (int e = 0; e < V; ++e) db[e] = dg[e] = 0.f;
    if (lane < lanes) {
        float a[V], b[V], m[V], rs[V], s1[V], s2[V], ga[V];
        affine<V>(A, n, c0, gamma, beta, mean, rstd, a, b, m, rs);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            ga[e] = gamma ? gamma[c0 + e] : 1.f;
            if (PASS == 1) {
                const float2 t = coef[n * A.groups + (c0 + e) / A.cg];
                s1[e] = t.x;
                s2[e] = t.y;
            }
        }
        for (int64_t r = r0 + lane; r < r1; r += lanes) {
            float g[V], best[V], f[V];
            int at[V];
            load<T, V>(dy + (n * A.total + r) * A.yp + c0, g);
            if (POOL == CF_POOL_MAX) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    load<T, V>(x + voxel_of<POOL>(A, n, r, k) + c0, f);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float u = fmaf(a[e], f[e] - m[e], b[e]);
                        if (k == 0 || u > best[e]) {
                            best[e] = u;
                            at[e] = k;
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < V; ++e) g[e] *= act_grad<ACT>(best[e], A.slope);
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float o[V];
                const int64_t vox = voxel_of<POOL>(A, n, r, k) + c0;
                load<T, V>(x + vox, f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float du;
                    if (POOL == CF_POOL_MAX)
                        du = at[e] == k ? g[e] : 0.f;
                    else
                        du = (POOL == CF_POOL_AVG ? 0.125f : 1.f) * g[e] * act_grad<ACT>(fmaf(a[e], f[e] - m[e], b[e]), A.slope);
                    const float xh = (f[e] - m[e]) * rs[e];
                    if (PASS == 0) {
                        db[e] += du;
                        dg[e] = fmaf(du, xh, dg[e]);
                    } else {
                        o[e] = rs[e] * (ga[e] * du - s1[e] - xh * s2[e]);
                    }
                }
                if (PASS == 1) store<T, V>(dx + vox, o);
            }
        }
    }
    if (PASS == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            sb[threadIdx.x * V + e] = db[e];
            sg[threadIdx.x * V + e] = dg[e];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < cols * V; i += kThreads) {
            float tb = 0.f, tg = 0.f;
            for (int l = 0; l < lanes; ++l) {
                tb += sb[(l * cols) * V + i];
                tg += sg[(l * cols) * V + i];
            }
            part[(n * A.chunks + blockIdx.x) * A.c + (int)blockIdx.y * kThreads * V + i] = make_float2(tb, tg);
        }
    }
}

// Blocks 0 .. n*groups-1: a group's means of gamma du and gamma du xh; the rest: dbeta and dgamma of 256 channels each.
__global__ void __launch_bounds__(kThreads) gn_bwd_reduce_kernel(GnArgs A, const float2* __restrict__ part,
                                                                const float* __restrict__ gamma, float2* __restrict__ coef,
                                                                float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ double red[kThreads / 32];
    const int64_t ng = A.n * A.groups;
    if (blockIdx.x < ng) {
        const int64_t n = blockIdx.x / A.groups;
        const int g = blockIdx.x % A.groups;
        double s1 = 0.0, s2 = 0.0;
        for (int i = threadIdx.x; i < A.chunks * A.cg; i += kThreads) {
            const int ch = i / A.cg, c = g * A.cg + i % A.cg;
            const float2 p = part[(n * A.chunks + ch) * A.c + c];
            const double ga = gamma ? gamma[c] : 1.f;
            s1 += ga * (double)p.x;
            s2 += ga * (double)p.y;
        }
        const double count = (double)A.s * A.cg;
        s1 = block_sum(s1, red);
        s2 = block_sum(s2, red);
        if (threadIdx.x == 0) coef[blockIdx.x] = make_float2((float)(s1 / count), (float)(s2 / count));
        return;
    }
    const int c = (int)(blockIdx.x - ng) * kThreads + threadIdx.x;
    if (c >= A.c) return;
    double tb = 0.0, tg = 0.0;
    for (int64_t i = 0; i < A.n * A.chunks; ++i) {
        const float2 p = part[i * A.c + c];
        tb += (double)p.x;
        tg += (double)p.y;
    }
    if (dbeta) dbeta[c] = (float)tb;
    if (dgamma) dgamma[c] = (float)tg;
}

bool desc_ok(const cf_gn_desc* d) {
    if (d == nullptr) return false;
    if (d->n <= 0 || d->d <= 0 || d->h <= 0 || d->w <= 0 || d->c <= 0 || d->groups <= 0) return false;
    if (d->c % d->groups != 0 || d->pool < CF_POOL_MAX || d->pool > CF_POOL_NONE) return false;
    if (d->act != CF_ACT_LRELU && d->act != CF_ACT_SILU) return false;
    if (d->dtype != CF_DT_BF16 && d->dtype != CF_DT_F32) return false;
    if (!(d->eps >= 0.f) || !(d->slope == d->slope)) return false;
    if ((d->x_pitch != 0 && d->x_pitch < d->c) || (d->y_pitch != 0 && d->y_pitch < d->c)) return false;
    if (d->d > (1 << 20) || d->h > (1 << 20) || d->w > (1 << 20) || d->n > 65535) return false;
    const double p = (double)std::max<int64_t>(std::max(d->x_pitch, d->y_pitch), d->c);
    return (double)d->n * d->d * d->h * d->w * p < 4.0e18;
}

cf_status supported(const cf_gn_desc* d) {
    if (d->pool != CF_POOL_NONE && (((d->d | d->h | d->w) & 1) || d->dtype != CF_DT_BF16)) return CF_ERR_UNSUPPORTED;
    if (d->pool == CF_POOL_MAX && (d->act != CF_ACT_LRELU || !(d->slope >= 0.f))) return CF_ERR_UNSUPPORTED;
    return CF_OK;
}

// Chunks of a sample: about four blocks of each pass to an SM, at least 32 rows a chunk.
GnArgs make_args(const cf_gn_desc* d, int num_sms, bool pooled_rows) {
    GnArgs A{};
    A.n = d->n, A.d = d->d, A.h = d->h, A.w = d->w, A.s = d->d * d->h * d->w;
    A.c = d->c, A.groups = d->groups, A.cg = d->c / d->groups;
    A.xp = d->x_pitch ? d->x_pitch : d->c, A.yp = d->y_pitch ? d->y_pitch : d->c;
    A.slope = d->slope, A.eps = d->eps;
    A.total = pooled_rows && d->pool != CF_POOL_NONE ? A.s / 8 : A.s;
    const int64_t want = std::max<int64_t>(1, 4 * num_sms / d->n);
    A.rows = std::max<int64_t>(32, (A.total + want - 1) / want);
    A.chunks = (int)((A.total + A.rows - 1) / A.rows);
    return A;
}

size_t part_bytes(const GnArgs& A) { return (size_t)A.n * A.chunks * A.c * sizeof(float2); }

// Values of a vector access: 16 bytes where channels, pitches and their alignment allow it, else one value.
int vec_of(const cf_gn_desc* d, const GnArgs& A) {
    const int v = d->dtype == CF_DT_F32 ? 4 : 8;
    return A.c % v == 0 && A.xp % v == 0 && A.yp % v == 0 ? v : 1;
}

dim3 grid_of(const GnArgs& A, int v) { return dim3(A.chunks, (A.c / v + kThreads - 1) / kThreads, (unsigned)A.n); }

template <typename T, int V>
cf_status forward(const LaunchCtx& ctx, const cf_gn_desc* d, const void* x, const float* gamma, const float* beta, void* y,
                  float* mean, float* rstd, float2* part) {
    const GnArgs S = make_args(d, ctx.num_sms, false), P = make_args(d, ctx.num_sms, true);
    const T* xt = static_cast<const T*>(x);
    T* yt = static_cast<T*>(y);
    gn_stats_kernel<T, V><<<grid_of(S, V), kThreads, 0, ctx.stream>>>(S, xt, part);
    gn_stats_reduce_kernel<<<(unsigned)(S.n * S.groups), kThreads, 0, ctx.stream>>>(S, part, mean, rstd);
#define CF_GN_APPLY(POOL, ACT) \
    gn_apply_kernel<T, V, POOL, ACT><<<grid_of(P, V), kThreads, 0, ctx.stream>>>(P, xt, gamma, beta, mean, rstd, yt)
    if (d->pool == CF_POOL_NONE) {
        if (d->act == CF_ACT_SILU)
            CF_GN_APPLY(CF_POOL_NONE, CF_ACT_SILU);
        else
            CF_GN_APPLY(CF_POOL_NONE, CF_ACT_LRELU);
    } else if constexpr (sizeof(T) == 2) {
        if (d->pool == CF_POOL_MAX)
            CF_GN_APPLY(CF_POOL_MAX, CF_ACT_LRELU);
        else if (d->act == CF_ACT_SILU)
            CF_GN_APPLY(CF_POOL_AVG, CF_ACT_SILU);
        else
            CF_GN_APPLY(CF_POOL_AVG, CF_ACT_LRELU);
    }
#undef CF_GN_APPLY
    return cudaGetLastError() == cudaSuccess ? CF_OK : CF_ERR_CUDA;
}

template <typename T, int V>
cf_status backward(const LaunchCtx& ctx, const cf_gn_desc* d, const void* x, const float* gamma, const float* beta,
                   const float* mean, const float* rstd, const void* dy, void* dx, float* dgamma, float* dbeta, float2* part,
                   float2* coef) {
    const GnArgs P = make_args(d, ctx.num_sms, true);
    const T *xt = static_cast<const T*>(x), *dyt = static_cast<const T*>(dy);
    T* dxt = static_cast<T*>(dx);
#define CF_GN_BWD(POOL, ACT, PASS)                                                                                        \
    gn_bwd_kernel<T, V, POOL, ACT, PASS>                                                                                  \
        <<<grid_of(P, V), kThreads, 0, ctx.stream>>>(P, xt, gamma, beta, mean, rstd, dyt, coef, part, dxt)
#define CF_GN_PASS(PASS)                                     \
    if (d->pool == CF_POOL_NONE) {                           \
        if (d->act == CF_ACT_SILU)                           \
            CF_GN_BWD(CF_POOL_NONE, CF_ACT_SILU, PASS);      \
        else                                                 \
            CF_GN_BWD(CF_POOL_NONE, CF_ACT_LRELU, PASS);     \
    } else if constexpr (sizeof(T) == 2) {                   \
        if (d->pool == CF_POOL_MAX)                          \
            CF_GN_BWD(CF_POOL_MAX, CF_ACT_LRELU, PASS);      \
        else if (d->act == CF_ACT_SILU)                      \
            CF_GN_BWD(CF_POOL_AVG, CF_ACT_SILU, PASS);       \
        else                                                 \
            CF_GN_BWD(CF_POOL_AVG, CF_ACT_LRELU, PASS);      \
    }
    CF_GN_PASS(0)
    gn_bwd_reduce_kernel<<<(unsigned)(P.n * P.groups + (P.c + kThreads - 1) / kThreads), kThreads, 0, ctx.stream>>>(
        P, part, gamma, coef, dgamma, dbeta);
    if (dx != nullptr) {
        CF_GN_PASS(1)
    }
#undef CF_GN_PASS
#undef CF_GN_BWD
    return cudaGetLastError() == cudaSuccess ? CF_OK : CF_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t workspace_bytes(const cf_gn_desc* d, int num_sms, bool backward) {
    const GnArgs A = make_args(d, num_sms, backward);
    return (size_t)A.n * A.groups * sizeof(float2) + 256 + part_bytes(A);
}

}  // namespace
}  // namespace cf

using namespace cf;

extern "C" {

size_t cf_group_norm_workspace_size(const cf_gn_desc* desc, int32_t backward) {
    if (!desc_ok(desc) || supported(desc) != CF_OK) return 0;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, nullptr)) return 0;
    return workspace_bytes(desc, ctx.num_sms, backward != 0);
}

cf_status cf_group_norm_fwd(const cf_gn_desc* desc, const void* x, const float* gamma, const float* beta, void* y,
                            float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream) {
    if (!desc_ok(desc) || x == nullptr || y == nullptr) return CF_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) || !aligned16(rstd) ||
        !aligned16(ws))
        return CF_ERR_INVALID_ARG;
    if (const cf_status st = supported(desc); st != CF_OK) return st;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    if (ws == nullptr || ws_bytes < workspace_bytes(desc, ctx.num_sms, false)) return CF_ERR_WORKSPACE;
    const GnArgs S = make_args(desc, ctx.num_sms, false);
    const size_t ng = (size_t)S.n * S.groups;
    if (mean == nullptr) mean = static_cast<float*>(ws);
    if (rstd == nullptr) rstd = static_cast<float*>(ws) + ng;
    float2* part = reinterpret_cast<float2*>(static_cast<char*>(ws) + (ng * sizeof(float2) + 255) / 256 * 256);
    if (desc->dtype == CF_DT_F32)
        return vec_of(desc, S) > 1 ? forward<float, 4>(ctx, desc, x, gamma, beta, y, mean, rstd, part)
                                   : forward<float, 1>(ctx, desc, x, gamma, beta, y, mean, rstd, part);
    return vec_of(desc, S) > 1 ? forward<uint16_t, 8>(ctx, desc, x, gamma, beta, y, mean, rstd, part)
                               : forward<uint16_t, 1>(ctx, desc, x, gamma, beta, y, mean, rstd, part);
}

cf_status cf_group_norm_bwd(const cf_gn_desc* desc, const void* x, const float* gamma, const float* beta,
                            const float* mean, const float* rstd, const void* dy, void* dx, float* dgamma,
                            float* dbeta, void* ws, size_t ws_bytes, void* stream) {
    if (!desc_ok(desc) || x == nullptr || mean == nullptr || rstd == nullptr || dy == nullptr) return CF_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(dy) || !aligned16(dx) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) ||
        !aligned16(rstd) || !aligned16(dgamma) || !aligned16(dbeta) || !aligned16(ws))
        return CF_ERR_INVALID_ARG;
    if (const cf_status st = supported(desc); st != CF_OK) return st;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    if (ws == nullptr || ws_bytes < workspace_bytes(desc, ctx.num_sms, true)) return CF_ERR_WORKSPACE;
    const GnArgs P = make_args(desc, ctx.num_sms, true);
    float2* coef = static_cast<float2*>(ws);
    float2* part =
        reinterpret_cast<float2*>(static_cast<char*>(ws) + ((size_t)P.n * P.groups * sizeof(float2) + 255) / 256 * 256);
    if (desc->dtype == CF_DT_F32)
        return vec_of(desc, P) > 1
                   ? backward<float, 4>(ctx, desc, x, gamma, beta, mean, rstd, dy, dx, dgamma, dbeta, part, coef)
                   : backward<float, 1>(ctx, desc, x, gamma, beta, mean, rstd, dy, dx, dgamma, dbeta, part, coef);
    return vec_of(desc, P) > 1
               ? backward<uint16_t, 8>(ctx, desc, x, gamma, beta, mean, rstd, dy, dx, dgamma, dbeta, part, coef)
               : backward<uint16_t, 1>(ctx, desc, x, gamma, beta, mean, rstd, dy, dx, dgamma, dbeta, part, coef);
}

}  // extern "C"
