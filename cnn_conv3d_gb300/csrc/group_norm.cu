// group_norm.cu -- group normalisation of NDHWC volumes with the block's
// activation and pooling, forward and backward, and their entry points.
//
// Each direction is a pass that sums over row chunks, a small kernel that adds
// the chunks up and makes the coefficients, and a pass that writes the output.
// Memory bounds both passes: a chunk is a few rows of every thread and one
// block's work, so that many blocks are resident and the ends of some lie under
// the loads of others.  The output pass goes backwards: what the sums read
// last, and L2 still has, it reads first.  (Persistent blocks that took chunks
// by a ticket were slower: each chunk then began with an atomic's and a load's
// latency.)  8 x 128^3 x 32 bf16 with max pooling, 1.07 GB in: 329 us, 6.9 TB/s
// of what is read twice and written once; the traffic that the algorithm cannot
// do without, x once, would take 181 us at the copy rate.
//
// Samples that a cluster's registers hold are read once, by one kernel
// (small_args): there a call is latency, 6 us for 8 x 4^3 x 256 forward and 8 us
// for 2 x 8^3 x 128 backward with the launch.
#include <cuda_bf16.h>

#include <algorithm>

#include "cf_internal.h"
#include "cf_ptx.cuh"
#include "fastdiv.cuh"

namespace cf {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct GnArgs {
    int64_t s;               // voxels of a sample
    int64_t xp, yp;
    int n, d, h, w, c, groups, cg;
    int tiles, tile;         // column tiles of `tile` vectors (the last may be narrower)
    float slope, eps;
    int chunks;              // row chunks of a sample, in both passes
    int srows, rows;         // voxels of a chunk in the statistics pass; voxels or windows of a chunk elsewhere
    int64_t total;           // voxels or windows of a sample
    FastDiv w2, h2, tdiv, cdiv, gdiv;  // pooled extents, tile, chunks, channels of a group
    float2* part;            // sums of a chunk
    float4* coef;            // [n][c]: (a, mean, beta, rstd)
    float2* lin;             // [n][c]: the backward's (k0, k1)
    float2* chan;            // [n][c]: the backward's channel sums of a sample
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

// V values of a voxel, as loaded.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
// Element by element, two at a time where the vector allows it.
template <int V>
__device__ __forceinline__ void vsub(float (&o)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 t = __fadd2_rn(make_float2(a[e], a[e + 1]), make_float2(-b[e], -b[e + 1]));
            o[e] = t.x, o[e + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = a[e] - b[e];
    }
}
template <int V>
__device__ __forceinline__ void vadd(float (&o)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 t = __fadd2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
            o[e] = t.x, o[e + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = a[e] + b[e];
    }
}
template <int V>
__device__ __forceinline__ void vfma(float (&o)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 t = __ffma2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), make_float2(c[e], c[e + 1]));
            o[e] = t.x, o[e + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(a[e], b[e], c[e]);
    }
}

template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& t, float (&f)[V]) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&t);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            f[2 * e] = __uint_as_float(w[e] << 16);
            f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = to_f<T>(t.v[e]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&f)[V]) {
    Pack<T, V> t;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&t);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) t.v[e] = from_f<T>(f[e]);
    }
    *reinterpret_cast<Pack<T, V>*>(p) = t;
}

// 1 / (1 + exp(-u)): to the last bits for fp32 outputs, by the fast exponential and division (relative error about
// 1e-6 at |u| of 10) where the result is rounded to bf16.
template <typename T>
__device__ __forceinline__ float sigmoid(float u) {
    if (sizeof(T) == 4) return 1.f / (1.f + expf(-u));
    return __fdividef(1.f, 1.f + __expf(-u));
}
template <typename T, int ACT>
__device__ __forceinline__ float act_of(float u, float slope) {
    if (ACT == CF_ACT_SILU) return u * sigmoid<T>(u);
    return u > 0.f ? u : slope * u;
}
template <typename T, int ACT>
__device__ __forceinline__ float act_grad(float u, float slope) {
    if (ACT == CF_ACT_SILU) {
        const float e = sigmoid<T>(u);
        return e * fmaf(u, 1.f - e, 1.f);
    }
    return u > 0.f ? 1.f : slope;
}

// Where a block works: its sample, columns and rows, and where a thread stands in them.
template <int V>
struct Place {
    int sample, chunk, tile;
    int64_t r0;               // first row
    int rows, cols, lanes, col, lane, c0, left;  // left: rows of the thread
    __device__ __forceinline__ Place(const GnArgs& A, int block, int per, int64_t total) {
        sample = (int)A.cdiv.div(block);
        chunk = block - sample * A.chunks;
        tile = blockIdx.y;
        r0 = (int64_t)chunk * per;
        rows = (int)min((int64_t)per, total - r0);
        if (A.tiles == 1) {
            cols = A.tile;
            lane = (int)A.tdiv.div(threadIdx.x);
        } else {
            cols = min(A.c / V - tile * A.tile, A.tile);
            lane = threadIdx.x / cols;
        }
        lanes = kThreads / cols;
        col = threadIdx.x - lane * cols;
        c0 = (tile * A.tile + col) * V;
        left = lane < lanes && rows > lane ? (int)((uint32_t)(rows - lane + lanes - 1) / (uint32_t)lanes) : 0;
    }
};

// The offset in x (in values) of a window's first voxel, and of the others from it.  A sample has fewer than 2^32 windows.
__device__ __forceinline__ int64_t window_at(const GnArgs& A, int64_t row) {
    const uint32_t m = (uint32_t)row, q = A.w2.div(m), pw = m - q * A.w2.d, pd = A.h2.div(q), ph = q - pd * A.h2.d;
    return (((int64_t)(2 * pd) * A.h + 2 * ph) * A.w + 2 * pw) * A.xp;
}
struct Window {
    int64_t d, h, w;
    __device__ __forceinline__ Window(const GnArgs& A) : d(A.xp * A.w * A.h), h(A.xp * A.w), w(A.xp) {}
    __device__ __forceinline__ int64_t at(int k) const { return (k & 4 ? d : 0) + (k & 2 ? h : 0) + (k & 1 ? w : 0); }
};

// A launch may begin while the one before it ends: it waits for that one's results here, and lets its own successor begin.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A sum of squares less what rounding took below 0; NaN stays NaN.
__device__ __forceinline__ float nonneg(float v) { return v < 0.f ? 0.f : v; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// A thread's own ring of 16-byte slots in shared memory, filled by asynchronous copies: the backward's passes have no registers
// for as many loads as must be in flight.  No thread waits for another's.
constexpr uint32_t kSlot = kThreads * 16;  // from a thread's slot to its next
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> slot(uint32_t at) {
    Pack<T, V> t;
    uint32_t* w = reinterpret_cast<uint32_t*>(&t);
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    return t;
}

// A thread's way through its rows of x (WIN: a window's eight voxels each) and dy, f(x's vectors, dy's) for each: through the
// ring where vectors are 16 bytes, two batches of rows ahead.
template <typename T, int V, bool WIN>
struct Rows {
    static constexpr int K = WIN ? 8 : 1, kBatch = WIN ? 1 : 4, kSlots = 2 * kBatch * (K + 1);
    static constexpr bool kRing = sizeof(T) * V == 16;
    static constexpr int kBytes = kRing ? kSlots * (int)kSlot : 0;
    const T *xs, *px, *pd;
    int64_t xstep, ystep, row;
    int step, left, ahead;
    Window w;

    __device__ __forceinline__ Rows(const GnArgs& A, const Place<V>& P, const T* x, const T* dy) : w(A) {
        xs = x + (int64_t)P.sample * A.s * A.xp + P.c0;
        row = P.r0 + P.lane;
        step = P.lanes;
        left = ahead = P.left;
        px = xs + (WIN ? window_at(A, row) : row * A.xp);
        pd = dy + ((int64_t)P.sample * A.total + row) * A.yp + P.c0;
        xstep = (int64_t)P.lanes * A.xp;
        ystep = (int64_t)P.lanes * A.yp;
    }
    __device__ __forceinline__ void next(const GnArgs& A) {
        row += step;
        px = WIN ? xs + window_at(A, row) : px + xstep;
        pd += ystep;
    }
    __device__ __forceinline__ void fetch(const GnArgs& A, uint32_t at) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (i < ahead) {
#pragma unroll
                for (int j = 0; j < K; ++j) copy16(at + (i * (K + 1) + j) * kSlot, px + (WIN ? w.at(j) : 0));
                copy16(at + (i * (K + 1) + K) * kSlot, pd);
                next(A);
            }
        copy_commit();
        ahead -= kBatch;
    }
    template <typename F>
    __device__ __forceinline__ void each(const GnArgs& A, uint32_t ring, F f) {
        if constexpr (kRing) {
            constexpr uint32_t kHalf = kBatch * (K + 1) * kSlot;
            fetch(A, ring);
            fetch(A, ring + kHalf);
            uint32_t at = ring;
            for (int i = 0; i < left; i += kBatch) {
                copy_wait<1>();
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (i + u < left) {
                        Pack<T, V> t[K];
#pragma unroll
                        for (int j = 0; j < K; ++j) t[j] = slot<T, V>(at + (u * (K + 1) + j) * kSlot);
                        f(t, slot<T, V>(at + (u * (K + 1) + K) * kSlot));
                    }
                fetch(A, at);
                at = at == ring ? ring + kHalf : ring;
            }
            copy_wait<0>();
        } else {
            constexpr int U = WIN ? 1 : 4;
            for (int i = 0; i < left; i += U) {
                Pack<T, V> t[U][K], d[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i + u < left) {
#pragma unroll
                        for (int j = 0; j < K; ++j) t[u][j] = load<T, V>(px + (WIN ? w.at(j) : 0));
                        d[u] = load<T, V>(pd);
                        next(A);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i + u < left) f(t[u], d[u]);
            }
        }
    }
};

// How a block adds up per group: a thread joins `span` neighbouring values of its vector, which are of one group, to a unit;
// a group is `units` units, a warp takes its units times the row lanes.
template <int V>
struct Span {
    int span, per, sh, units;  // per = 1 << sh: units of a vector
    __device__ __forceinline__ Span(const GnArgs& A) {
        span = A.cg % V == 0 ? V : V % A.cg == 0 ? A.cg : 1;
        per = V / span;
        sh = 31 - __clz(per);
        units = A.cg / span;
    }
};
// Calls f(entry, row lane) for the entries of group g that the block's column tile has, shared out over a warp; an entry is
// at [unit of the vector][thread].  Returns their number of units.
template <int V, typename F>
__device__ __forceinline__ int group_entries(const GnArgs& A, const Place<V>& P, const Span<V>& sp, int g, F f) {
    const int at0 = P.tile * A.tile * sp.per, wide = P.cols * sp.per;  // units
    const int qa = max(g * sp.units - at0, 0), qb = min((g + 1) * sp.units - at0, wide);
    const int lane = threadIdx.x & 31;
    int lp = 32, sh = 5;  // lanes of the warp that take row lanes; the others take further units
    while (lp > P.lanes) lp >>= 1, --sh;
    for (int q = qa + (lane >> sh); q < qb; q += 32 >> sh) {
        const int col = q >> sp.sh, slot = q & (sp.per - 1);
        for (int l = lane & (lp - 1); l < P.lanes; l += lp) f(slot * kThreads + l * P.cols + col, l);
    }
    return qb - qa;
}

// Mean and sum of squared deviations of each group over a chunk: part[sample][chunk][tile][group].  A thread sums about its
// first row, then about the mean of its first few: where the first row is far off, no more than a factor of those few can be
// lost in the rounding.  DRAM reads bound it: 157 us for 1.07 GB, 6.9 TB/s, with eight 16-byte loads of a thread in flight and
// three blocks an SM (with four loads both passes took 334 us, with eight 329).
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 3) gn_stats_kernel(const GnArgs A, const T* __restrict__ x) {
    __shared__ float sm[kThreads * V], sq[kThreads * V];
    grid_go();
    const Place<V> P(A, blockIdx.x, A.srows, A.s);
    float k[V], s[V], q[V];
#pragma unroll
    for (int e = 0; e < V; ++e) k[e] = s[e] = q[e] = 0.f;
    if (P.left) {
        constexpr int U = 8;
        const int64_t step = (int64_t)P.lanes * A.xp;
        const T* p = x + ((int64_t)P.sample * A.s + P.r0 + P.lane) * A.xp + P.c0;
        unpack<T, V>(load<T, V>(p), k);
        auto add = [&](const Pack<T, V>& t) {
            float f[V];
            unpack<T, V>(t, f);
            vsub<V>(f, f, k);
            vadd<V>(s, s, f);
            vfma<V>(q, f, f, q);
        };
        // the sums moved from about k to about the mean of the n rows so far
        auto recentre = [&](int n) {
            const float inv = 1.f / (float)n;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = s[e] * inv;
                k[e] += d;
                q[e] = nonneg(fmaf(-s[e], d, q[e]));
                s[e] = 0.f;
            }
        };
        int i = P.left;
        for (; i >= U; i -= U, p += U * step) {
            Pack<T, V> t[U];
#pragma unroll
            for (int u = 0; u < U; ++u) t[u] = load<T, V>(p + u * step);
#pragma unroll
            for (int u = 0; u < U; ++u) add(t[u]);
            if (i == P.left) recentre(U);
        }
        for (; i > 0; --i, p += step) add(load<T, V>(p));
        recentre(P.left);
    }
    const Span<V> sp(A);
    // neighbours of equal counts: the mean of their means, and the deviations from it
#pragma unroll
    for (int w = 1; w < V; w *= 2)
        if (w < sp.span) {
#pragma unroll
            for (int e = 0; e + w < V; e += 2 * w) {
                const float d = k[e + w] - k[e];
                k[e] = fmaf(0.5f, d, k[e]);
                q[e] += fmaf(0.5f * (float)(w * P.left) * d, d, q[e + w]);
            }
        }
#pragma unroll
    for (int e = 0; e < V; ++e)
        if ((e & (sp.span - 1)) == 0) {
            const int at = (e * sp.per / V) * kThreads + threadIdx.x;
            sm[at] = k[e];
            sq[at] = q[e];
        }
    __syncthreads();
    // a warp to a group: sums about the mean of its first entry
    const int first = P.tile * A.tile * V, g0 = first / A.cg, g1 = (first + P.cols * V - 1) / A.cg;
    const int least = P.rows / P.lanes, more = P.rows - least * P.lanes;  // rows of a lane: least, or one more
    for (int g = g0 + (threadIdx.x >> 5); g <= g1; g += kWarps) {
        const int q0 = max(g * sp.units - P.tile * A.tile * sp.per, 0);
        const float about = sm[(q0 & (sp.per - 1)) * kThreads + (q0 >> sp.sh)];
        float a = 0.f, b = 0.f;
        const int units = group_entries<V>(A, P, sp, g, [&](int at, int l) {
            const float nl = (float)((least + (l < more)) * sp.span), d = sm[at] - about;
            a = fmaf(nl, d, a);
            b += nl > 0.f ? fmaf(nl * d, d, sq[at]) : 0.f;
        });
        a = warp_sum(a);
        b = warp_sum(b);
        const float d = a / ((float)P.rows * (float)(units * sp.span));
        if ((threadIdx.x & 31) == 0)
            A.part[((int64_t)blockIdx.x * A.tiles + P.tile) * A.groups + g] = make_float2(about + d, nonneg(fmaf(-a, d, b)));
    }
}

// Channels of group g in column tile t.
template <int V>
__device__ __forceinline__ int channels_in(const GnArgs& A, int g, int t) {
    const int b = t * A.tile * V, e = min(b + A.tile * V, A.c);
    return max(min((g + 1) * A.cg, e) - max(g * A.cg, b), 0);
}

__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t += red[i];
    return t;
}

// Mean and rstd of a group from the chunks' statistics, a block to a group, and the coefficients of its channels.  4 to 6 us, all
// latency, most of it under the end of the statistics pass.
template <int V>
__global__ void __launch_bounds__(kThreads) gn_finish_kernel(const GnArgs A, const float* __restrict__ gamma,
                                                            const float* __restrict__ beta, float* __restrict__ mean,
                                                            float* __restrict__ rstd) {
    __shared__ float red[kWarps];
    grid_go();
    grid_wait();
    const int sample = blockIdx.x / A.groups, g = blockIdx.x - sample * A.groups, items = A.chunks * A.tiles;
    const float2* p = A.part + (int64_t)sample * items * A.groups + g;
    const float count = (float)A.s * (float)A.cg;
    auto weight = [&](int i) {
        const int ch = A.tiles == 1 ? i : i / A.tiles, nc = A.tiles == 1 ? A.cg : channels_in<V>(A, g, i - ch * A.tiles);
        return (float)min((int64_t)A.srows, A.s - (int64_t)ch * A.srows) * (float)nc;
    };
    // the first pass's values stay in registers for the second where a thread has no more than eight
    constexpr int kKeep = 8;
    float2 v[kKeep];
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
        const int i = threadIdx.x + u * kThreads;
        v[u] = i < items && weight(i) > 0.f ? p[(int64_t)i * A.groups] : make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
        const int i = threadIdx.x + u * kThreads;
        if (i < items && weight(i) > 0.f) s = fmaf(weight(i), v[u].x, s);
    }
    for (int i = threadIdx.x + kKeep * kThreads; i < items; i += kThreads)
        if (weight(i) > 0.f) s = fmaf(weight(i), p[(int64_t)i * A.groups].x, s);
    const float mu = block_sum(s, red) / count;
    float q = 0.f;
    auto dev = [&](int i, float2 t) {
        const float d = t.x - mu;
        q += fmaf(weight(i) * d, d, t.y);
    };
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
        const int i = threadIdx.x + u * kThreads;
        if (i < items && weight(i) > 0.f) dev(i, v[u]);
    }
    for (int i = threadIdx.x + kKeep * kThreads; i < items; i += kThreads)
        if (weight(i) > 0.f) dev(i, p[(int64_t)i * A.groups]);
    const float rs = 1.f / sqrtf(block_sum(q, red) / count + A.eps);
    if (threadIdx.x == 0) {
        if (mean) mean[blockIdx.x] = mu;
        if (rstd) rstd[blockIdx.x] = rs;
    }
    for (int i = threadIdx.x; i < A.cg; i += kThreads) {
        const int c = g * A.cg + i;
        A.coef[(int64_t)sample * A.c + c] = make_float4((gamma ? gamma[c] : 1.f) * rs, mu, beta ? beta[c] : 0.f, rs);
    }
}

// What the launch before wrote is read by plain loads: the read-only path is for data that nobody writes while the kernel runs, and
// this one may have begun before.
template <int V>
__device__ __forceinline__ void load_coef(const GnArgs& A, const Place<V>& P, float (&a)[V], float (&m)[V], float (&be)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float4 t = A.coef[(int64_t)P.sample * A.c + P.c0 + e];
        a[e] = t.x, m[e] = t.y, be[e] = t.z;
    }
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// The value among eight voxels that maximises u = a (x - mean) + beta: the maximum, or for a < 0 the minimum, taken on packed
// bf16 with the sign bits of such channels flipped.
template <typename T, int V>
__device__ __forceinline__ void window_max(const Pack<T, V>* t, const float (&a)[V], float (&best)[V]) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            const uint32_t flip = (a[2 * e] < 0.f ? 0x8000u : 0u) | (a[2 * e + 1] < 0.f ? 0x80000000u : 0u);
            uint32_t m = reinterpret_cast<const uint32_t*>(&t[0])[e] ^ flip;
#pragma unroll
            for (int k = 1; k < 8; ++k) m = max_bf16x2(m, reinterpret_cast<const uint32_t*>(&t[k])[e] ^ flip);
            m ^= flip;
            best[2 * e] = __uint_as_float(m << 16);
            best[2 * e + 1] = __uint_as_float(m & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            best[e] = to_f<T>(t[0].v[e]);
#pragma unroll
            for (int k = 1; k < 8; ++k) {
                const float f = to_f<T>(t[k].v[e]);
                best[e] = a[e] < 0.f ? fminf(best[e], f) : fmaxf(best[e], f);
            }
        }
    }
    // a = 0: every voxel's u is beta, and the first is the maximum
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (a[e] == 0.f) best[e] = to_f<T>(t[0].v[e]);
}

// The output of a chunk.  DRAM bounds it: 174 us for 1.07 GB in and 134 MB out (8 x 128^3 x 32, max pooling), 6.9 TB/s.
template <typename T, int V, int POOL, int ACT>
__global__ void __launch_bounds__(kThreads, POOL == CF_POOL_NONE ? 4 : 3) gn_apply_kernel(const GnArgs A, const T* __restrict__ x,
                                                                                       T* __restrict__ y) {
    const Place<V> P(A, gridDim.x - 1 - blockIdx.x, A.rows, A.total);
    grid_wait();
    if (!P.left) return;
    float a[V], m[V], be[V];
    load_coef<V>(A, P, a, m, be);
    const T* xs = x + (int64_t)P.sample * A.s * A.xp + P.c0;
    T* o = y + ((int64_t)P.sample * A.total + P.r0 + P.lane) * A.yp + P.c0;
    const int64_t ystep = (int64_t)P.lanes * A.yp;
    auto norm = [&](float (&f)[V]) {
        vsub<V>(f, f, m);
        vfma<V>(f, a, f, be);
    };
    if constexpr (POOL == CF_POOL_NONE) {
        constexpr int U = V > 2 ? 4 : 8;
        const int64_t xstep = (int64_t)P.lanes * A.xp;
        const T* p = xs + (P.r0 + P.lane) * A.xp;
        auto one = [&](const Pack<T, V>& t, T* at) {
            float f[V];
            unpack<T, V>(t, f);
            norm(f);
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = act_of<T, ACT>(f[e], A.slope);
            store<T, V>(at, f);
        };
        int i = P.left;
        for (; i >= U; i -= U, p += U * xstep, o += U * ystep) {
            Pack<T, V> t[U];
#pragma unroll
            for (int u = 0; u < U; ++u) t[u] = load<T, V>(p + u * xstep);
#pragma unroll
            for (int u = 0; u < U; ++u) one(t[u], o + u * ystep);
        }
        for (; i > 0; --i, p += xstep, o += ystep) one(load<T, V>(p), o);
    } else {
        const Window W(A);
        int64_t row = P.r0 + P.lane;
        for (int i = 0; i < P.left; ++i, row += P.lanes, o += ystep) {
            const T* p = xs + window_at(A, row);
            Pack<T, V> t[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) t[q] = load<T, V>(p + W.at(q));
            float f[V];
            if (POOL == CF_POOL_MAX) {
                window_max<T, V>(t, a, f);
                norm(f);
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = act_of<T, ACT>(f[e], A.slope);
            } else {
                float sum[V];
#pragma unroll
                for (int e = 0; e < V; ++e) sum[e] = 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    unpack<T, V>(t[q], f);
                    norm(f);
#pragma unroll
                    for (int e = 0; e < V; ++e) sum[e] += act_of<T, ACT>(f[e], A.slope);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = 0.125f * sum[e];
            }
            store<T, V>(o, f);
        }
    }
}

// Coefficients of the backward, [n][c], from the forward's statistics.
__global__ void __launch_bounds__(kThreads) gn_coef_kernel(const GnArgs A, const float* __restrict__ gamma,
                                                          const float* __restrict__ beta, const float* __restrict__ mean,
                                                          const float* __restrict__ rstd) {
    const int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    grid_go();
    if (i >= (int64_t)A.n * A.c) return;
    const int64_t n = i / A.c;
    const int c = (int)(i - n * A.c);
    const int64_t g = n * A.groups + c / A.cg;
    const float rs = rstd[g];
    A.coef[i] = make_float4((gamma ? gamma[c] : 1.f) * rs, mean[g], beta ? beta[c] : 0.f, rs);
}

// Channel sums of du and du xh over a chunk: part[sample][chunk][c].  x and dy come through a ring in shared memory of which each
// thread fills and reads its own part, so that no barrier holds the loads up.  8 x 64^3 x 64 with max pooling: 53 us for 302 MB,
// 5.7 TB/s.  Where x's rows are 96 bytes of each 224, DRAM is read in pieces that make 192 of them: 45 us for 248 MB, 165 wanted.
template <typename T, int V, int POOL, int ACT>
__global__ void __launch_bounds__(kThreads, 2) gn_bwd_sums_kernel(const GnArgs A, const T* __restrict__ x,
                                                                                          const T* __restrict__ dy) {
    extern __shared__ __align__(16) uint8_t ring[];  // afterwards the threads' sums
    const Place<V> P(A, blockIdx.x, A.rows, A.total);
    grid_go();
    grid_wait();
    float db[V], dg[V];
#pragma unroll
    for (int e = 0; e < V; ++e) db[e] = dg[e] = 0.f;
    if (P.left) {
        float a[V], m[V], be[V];
        load_coef<V>(A, P, a, m, be);
        auto add = [&](float (&f)[V], float (&g)[V]) {
            float u[V];
            vsub<V>(f, f, m);
            vfma<V>(u, a, f, be);
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] = g[e] * act_grad<T, ACT>(u[e], A.slope);
            vadd<V>(db, db, u);
            vfma<V>(dg, u, f, dg);
        };
        Rows<T, V, POOL != CF_POOL_NONE> W(A, P, x, dy);
        W.each(A, smem_u32(ring) + threadIdx.x * 16, [&](const auto& t, const Pack<T, V>& td) {
            float f[V], g[V];
            unpack<T, V>(td, g);
            if constexpr (POOL == CF_POOL_AVG) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    unpack<T, V>(td, g);
#pragma unroll
                    for (int e = 0; e < V; ++e) g[e] *= 0.125f;
                    unpack<T, V>(t[j], f);
                    add(f, g);
                }
            } else {
                if constexpr (POOL == CF_POOL_MAX)
                    window_max<T, V>(t, a, f);
                else
                    unpack<T, V>(t[0], f);
                add(f, g);
            }
        });
#pragma unroll
        for (int e = 0; e < V; ++e) dg[e] *= A.coef[(int64_t)P.sample * A.c + P.c0 + e].w;
    }
    float *sb = reinterpret_cast<float*>(ring), *sg = sb + kThreads * V;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) {
        sb[e * kThreads + threadIdx.x] = db[e];
        sg[e * kThreads + threadIdx.x] = dg[e];
    }
    __syncthreads();
    // a channel's row lanes are added up by as many neighbouring threads as the block has for it
    const int wide = P.cols * V;
    float2* part = A.part + (int64_t)blockIdx.x * A.c + P.tile * A.tile * V;
    int lp = 1;
    while (2 * lp <= 32 && 2 * lp <= P.lanes && 2 * lp * wide <= kThreads) lp *= 2;
    for (int i = threadIdx.x / lp; i < (wide + 31) / 32 * 32; i += kThreads / lp) {  // whole warps, for the shuffles
        float tb = 0.f, tg = 0.f;
        if (i < wide)
            for (int l = threadIdx.x & (lp - 1); l < P.lanes; l += lp) {
                tb += sb[i % V * kThreads + l * P.cols + i / V];
                tg += sg[i % V * kThreads + l * P.cols + i / V];
            }
        for (int o = lp / 2; o; o >>= 1) {
            tb += __shfl_xor_sync(~0u, tb, o);
            tg += __shfl_xor_sync(~0u, tg, o);
        }
        if (i < wide && (threadIdx.x & (lp - 1)) == 0) part[i] = make_float2(tb, tg);
    }
}

// A group's channel sums from the chunks', a block to a group of a sample, and the rest of dx's coefficients:
// dx = a du + k1 (x - mean) + k0 with k0 = -rstd s1, k1 = -rstd^2 s2, s1 and s2 the group's means of gamma du and gamma du xh.
__global__ void __launch_bounds__(kThreads) gn_bwd_finish_kernel(const GnArgs A, const float* __restrict__ gamma) {
    __shared__ float2 red[kThreads];
    __shared__ float rw[kWarps];
    grid_go();
    grid_wait();
    const int sample = blockIdx.x / A.groups, g = blockIdx.x - sample * A.groups;
    const float2* p = A.part + (int64_t)sample * A.chunks * A.c + g * A.cg;
    const int64_t base = (int64_t)sample * A.c + g * A.cg;
    float s1 = 0.f, s2 = 0.f;
    for (int c0 = 0; c0 < A.cg; c0 += kThreads) {
        const int cols = min(A.cg - c0, kThreads), lanes = kThreads / cols, lane = threadIdx.x / cols, col = threadIdx.x - lane * cols;
        float tb = 0.f, tg = 0.f;
        if (lane < lanes) {
#pragma unroll 8
            for (int i = lane; i < A.chunks; i += lanes) {
                const float2 v = p[(int64_t)i * A.c + c0 + col];
                tb += v.x;
                tg += v.y;
            }
        }
        __syncthreads();
        red[threadIdx.x] = make_float2(tb, tg);
        __syncthreads();
        // the lanes of a column in turn by halves
        for (int have = lanes; have > 1; have = (have + 1) / 2) {
            const int half = (have + 1) / 2;
            float2 t = red[threadIdx.x];
            if (lane < have - half) {
                const float2 u = red[threadIdx.x + half * cols];
                t.x += u.x, t.y += u.y;
                red[threadIdx.x] = t;
            }
            __syncthreads();
        }
        if (lane == 0) {
            const float2 t = red[col];
            A.chan[base + c0 + col] = t;
            const float ga = gamma ? gamma[g * A.cg + c0 + col] : 1.f;
            s1 = fmaf(ga, t.x, s1);
            s2 = fmaf(ga, t.y, s2);
        }
    }
    const float inv = 1.f / ((float)A.s * (float)A.cg), rs = A.coef[base].w;
    const float k0 = -rs * (block_sum(s1, rw) * inv), k1 = -rs * rs * (block_sum(s2, rw) * inv);
    for (int i = threadIdx.x; i < A.cg; i += kThreads) A.lin[base + i] = make_float2(k0, k1);
}

// dx of a chunk; the blocks from `work` on add up the samples' channel sums instead: dbeta, dgamma.  8 x 64^3 x 64 with max
// pooling: 90 us for 302 MB in and 268 MB out, 6.3 TB/s.
template <typename T, int V, int POOL, int ACT>
__global__ void __launch_bounds__(kThreads, 2) gn_bwd_apply_kernel(const GnArgs A, const T* __restrict__ x, const T* __restrict__ dy,
                                                                  T* __restrict__ dx, int work, float* __restrict__ dgamma,
                                                                  float* __restrict__ dbeta) {
    grid_wait();
    if ((int)blockIdx.x >= work) {
        const int c = ((int)blockIdx.x - work) * kThreads + threadIdx.x;
        if (blockIdx.y != 0 || c >= A.c) return;
        float tb = 0.f, tg = 0.f;
#pragma unroll 8
        for (int i = 0; i < A.n; ++i) {
            const float2 v = A.chan[(int64_t)i * A.c + c];
            tb += v.x;
            tg += v.y;
        }
        if (dbeta) dbeta[c] = tb;
        if (dgamma) dgamma[c] = tg;
        return;
    }
    const Place<V> P(A, work - 1 - blockIdx.x, A.rows, A.total);
    if (!P.left) return;
    float a[V], m[V], be[V], k0[V], k1[V];
    load_coef<V>(A, P, a, m, be);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float2 t = A.lin[(int64_t)P.sample * A.c + P.c0 + e];
        k0[e] = t.x, k1[e] = t.y;
    }
    extern __shared__ __align__(16) uint8_t ring[];
    Rows<T, V, POOL != CF_POOL_NONE> W(A, P, x, dy);
    T* os = dx + (int64_t)P.sample * A.s * A.xp + P.c0;
    int64_t row = P.r0 + P.lane;
    W.each(A, smem_u32(ring) + threadIdx.x * 16, [&](const auto& t, const Pack<T, V>& td) {
        T* o = os + (POOL == CF_POOL_NONE ? row * A.xp : window_at(A, row));
        row += P.lanes;
        float f[V], g[V], u[V];
        unpack<T, V>(td, g);
        if constexpr (POOL == CF_POOL_NONE) {
            unpack<T, V>(t[0], f);
            vsub<V>(f, f, m);
            vfma<V>(u, a, f, be);
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] *= act_grad<T, ACT>(u[e], A.slope);
            vfma<V>(f, k1, f, k0);
            vfma<V>(f, a, g, f);
            store<T, V>(o, f);
        } else {
            float best[V];
            if (POOL == CF_POOL_MAX) {
                window_max<T, V>(t, a, best);
                vsub<V>(u, best, m);
                vfma<V>(u, a, u, be);
#pragma unroll
                for (int e = 0; e < V; ++e) g[e] *= a[e] * act_grad<T, ACT>(u[e], A.slope);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) g[e] *= 0.125f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float lin[V];
                unpack<T, V>(t[j], f);
                vsub<V>(u, f, m);
                vfma<V>(lin, k1, u, k0);
                if (POOL == CF_POOL_MAX) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        // the first voxel that has the maximum takes the gradient and leaves none
                        const bool hit = f[e] == best[e];
                        lin[e] += hit ? g[e] : 0.f;
                        g[e] = hit ? 0.f : g[e];
                    }
                } else {
                    vfma<V>(u, a, u, be);
#pragma unroll
                    for (int e = 0; e < V; ++e) u[e] = g[e] * act_grad<T, ACT>(u[e], A.slope);
                    vfma<V>(lin, a, u, lin);
                }
                store<T, V>(o + W.w.at(j), lin);
            }
        }
    });
}

// ---------------------------------------------------------------------------
// Small samples: a cluster of blocks holds a sample's channels (or a part of them that is whole groups) in registers, so that
// one launch reads x (and dy) once; the blocks exchange their group sums through each other's shared memory.

constexpr int kSmallThreads = 256;
constexpr int kSmallWarps = kSmallThreads / 32;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A block of a cluster may only be written to once it has begun: cluster_begin where a block does, cluster_begun before its first
// store_remote.  The barrier's time lies under the loads between them.
__device__ __forceinline__ void cluster_begin() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores v at `at` (an address of this block's shared memory) in the block `rank` of the cluster.
__device__ __forceinline__ void store_remote(const float2* at, uint32_t rank, float2 v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

// Where a block of a cluster works: rows r0 .. r0+rows-1 of a sample, columns of tile blockIdx.y.
template <int V>
struct SmallPlace {
    int sample, rank, r0, rows, lanes, col, lane, c0, left;
    __device__ __forceinline__ SmallPlace(const GnArgs& A) {
        rank = (int)cluster_rank();
        sample = blockIdx.x / A.chunks;
        r0 = rank * A.rows;
        rows = max(0, min(A.rows, (int)A.total - r0));
        lane = (int)A.tdiv.div(threadIdx.x);
        lanes = kSmallThreads / A.tile;
        col = threadIdx.x - lane * A.tile;
        c0 = (blockIdx.y * A.tile + col) * V;
        left = lane < lanes && rows > lane ? (int)((uint32_t)(rows - lane + lanes - 1) / (uint32_t)lanes) : 0;
    }
};

// The thread's R items (a voxel's vector, or a window's eight) in registers.
template <typename T, int V, int POOL, int R>
struct Held {
    static constexpr int K = POOL == CF_POOL_NONE ? 1 : 8;
    Pack<T, V> t[R][K];
    __device__ __forceinline__ void load_all(const GnArgs& A, const SmallPlace<V>& P, const T* x) {
        const Window W(A);
        const T* xs = x + (int64_t)P.sample * A.s * A.xp + P.c0;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i < P.left) {
                const int64_t row = P.r0 + P.lane + i * P.lanes;
                const T* p = xs + (K == 1 ? row * A.xp : window_at(A, row));
#pragma unroll
                for (int k = 0; k < K; ++k) t[i][k] = load<T, V>(p + (K == 1 ? 0 : W.at(k)));
            }
    }
};

// Sums of the entries of the tile's group g (numbered from 0), over a warp: f(entry, row lane), an entry at
// [unit of the vector][thread].
template <int V, typename F>
__device__ __forceinline__ void small_entries(const GnArgs& A, int lanes, const Span<V>& sp, int g, F f) {
    const int lane = threadIdx.x & 31, qb = (g + 1) * sp.units;
    int lp = 32, sh = 5;
    while (lp > lanes) lp >>= 1, --sh;
    for (int q = g * sp.units + (lane >> sh); q < qb; q += 32 >> sh) {
        const int col = q >> sp.sh, slot = q & (sp.per - 1);
        for (int l = lane & (lp - 1); l < lanes; l += lp) f(slot * kSmallThreads + l * A.tile + col, l);
    }
}

// Forward of a sample's columns by a cluster that holds them in registers: x is read once, all of a thread's loads in flight, and
// the blocks exchange their groups' means and deviations through shared memory.  Latency bounds it: loads, two sums over the
// block, the cluster's barrier, stores.  8 x 4^3 x 256 bf16: 4.8 us by two blocks a sample's column, 5.2 by four, 6.2 by eight.
template <typename T, int V, int POOL, int ACT, int R>
__global__ void __launch_bounds__(kSmallThreads, 2) gn_small_fwd_kernel(const GnArgs A, const T* __restrict__ x,
                                                                       const float* __restrict__ gamma, const float* __restrict__ beta,
                                                                       T* __restrict__ y, float* __restrict__ mean,
                                                                       float* __restrict__ rstd) {
    extern __shared__ float2 ex[];  // [rank][group of the tile], then the tile's (mean, rstd)
    __shared__ float sm[kSmallThreads * V], sq[kSmallThreads * V];
    cluster_begin();
    const SmallPlace<V> P(A);
    const int groups = A.tile * V / A.cg, g0 = blockIdx.y * groups;
    Held<T, V, POOL, R> H;
    H.load_all(A, P, x);
    float a[V], m[V], be[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        a[e] = gamma && P.left ? gamma[P.c0 + e] : 1.f;
        be[e] = beta && P.left ? beta[P.c0 + e] : 0.f;
    }
    float k[V], s[V], q[V];
#pragma unroll
    for (int e = 0; e < V; ++e) k[e] = s[e] = q[e] = 0.f;
    if (P.left) unpack<T, V>(H.t[0][0], k);
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < P.left) {
#pragma unroll
            for (int j = 0; j < H.K; ++j) {
                float f[V];
                unpack<T, V>(H.t[i][j], f);
                vsub<V>(f, f, k);
                vadd<V>(s, s, f);
                vfma<V>(q, f, f, q);
            }
        }
    const float n = (float)(P.left * H.K), inv = P.left ? 1.f / n : 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float d = s[e] * inv;
        k[e] += d;
        q[e] = nonneg(fmaf(-s[e], d, q[e]));
    }
    const Span<V> sp(A);
#pragma unroll
    for (int w = 1; w < V; w *= 2)
        if (w < sp.span) {
#pragma unroll
            for (int e = 0; e + w < V; e += 2 * w) {
                const float d = k[e + w] - k[e];
                k[e] = fmaf(0.5f, d, k[e]);
                q[e] += fmaf(0.5f * (float)w * n * d, d, q[e + w]);
            }
        }
#pragma unroll
    for (int e = 0; e < V; ++e)
        if ((e & (sp.span - 1)) == 0) {
            const int at = (e * sp.per / V) * kSmallThreads + threadIdx.x;
            sm[at] = k[e];
            sq[at] = q[e];
        }
    __syncthreads();
    cluster_begun();
    const int least = P.rows / P.lanes, more = P.rows - least * P.lanes;
    for (int g = threadIdx.x >> 5; g < groups; g += kSmallWarps) {
        const int q0 = g * sp.units;
        const float about = sm[(q0 & (sp.per - 1)) * kSmallThreads + (q0 >> sp.sh)];
        float sa = 0.f, sd = 0.f;
        small_entries<V>(A, P.lanes, sp, g, [&](int at, int l) {
            const float nl = (float)((least + (l < more)) * H.K * sp.span), d = sm[at] - about;
            sa = fmaf(nl, d, sa);
            sd += nl > 0.f ? fmaf(nl * d, d, sq[at]) : 0.f;
        });
        sa = warp_sum(sa);
        sd = warp_sum(sd);
        const float d = P.rows ? sa / ((float)(P.rows * H.K) * (float)A.cg) : 0.f;
        if ((threadIdx.x & 31) < A.chunks)
            store_remote(&ex[P.rank * groups + g], threadIdx.x & 31, make_float2(about + d, nonneg(fmaf(-sa, d, sd))));
    }
    cluster_sync();
    float2* stat = ex + A.chunks * groups;
    for (int g = threadIdx.x; g < groups; g += kSmallThreads) {
        // the blocks' means and deviations joined about the first's
        const float about = ex[g].x, per = (float)(H.K * A.cg);
        float sa = 0.f, sd = 0.f;
        for (int r = 0; r < A.chunks; ++r) {
            const float nr = (float)max(0, min(A.rows, (int)A.total - r * A.rows)) * per;
            const float2 t = ex[r * groups + g];
            const float d = t.x - about;
            if (nr > 0.f) {
                sa = fmaf(nr, d, sa);
                sd += fmaf(nr * d, d, t.y);
            }
        }
        const float count = (float)A.s * (float)A.cg, d = sa / count;
        const float mu = about + d, rs = 1.f / sqrtf(nonneg(fmaf(-sa, d, sd)) / count + A.eps);
        stat[g] = make_float2(mu, rs);
        if (P.rank == 0) {
            if (mean) mean[(int64_t)P.sample * A.groups + g0 + g] = mu;
            if (rstd) rstd[(int64_t)P.sample * A.groups + g0 + g] = rs;
        }
    }
    __syncthreads();
    if (!P.left) return;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float2 t = stat[A.gdiv.div(P.col * V + e)];
        m[e] = t.x;
        a[e] *= t.y;
    }
    auto norm = [&](float (&f)[V]) {
        vsub<V>(f, f, m);
        vfma<V>(f, a, f, be);
    };
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < P.left) {
            float f[V], o[V];
            if (POOL == CF_POOL_AVG) {
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = 0.f;
#pragma unroll
                for (int j = 0; j < H.K; ++j) {
                    unpack<T, V>(H.t[i][j], f);
                    norm(f);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += 0.125f * act_of<T, ACT>(f[e], A.slope);
                }
            } else {
                if constexpr (POOL == CF_POOL_MAX)
                    window_max<T, V>(H.t[i], a, o);
                else
                    unpack<T, V>(H.t[i][0], o);
                norm(o);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = act_of<T, ACT>(o[e], A.slope);
            }
            store<T, V>(y + ((int64_t)P.sample * A.total + P.r0 + P.lane + i * P.lanes) * A.yp + P.c0, o);
        }
}

// dx, and the block's channel sums: part[sample][rank][c].  2 x 8^3 x 128 bf16: 5.5 us by clusters of eight, 5.8 by four, 8.1 by
// two, 10 by one block, then 2.5 for the channels' sums.
template <typename T, int V, int POOL, int ACT, int R>
__global__ void __launch_bounds__(kSmallThreads, 2) gn_small_bwd_kernel(const GnArgs A, const T* __restrict__ x,
                                                                       const float* __restrict__ gamma, const float* __restrict__ beta,
                                                                       const float* __restrict__ mean, const float* __restrict__ rstd,
                                                                       const T* __restrict__ dy, T* __restrict__ dx) {
    extern __shared__ float2 ex[];  // [rank][group of the tile], then the tile's (s1, s2)
    grid_go();
    __shared__ float sb[kSmallThreads * V], sg[kSmallThreads * V];
    if (dx) cluster_begin();  // the same for the whole grid
    const SmallPlace<V> P(A);
    const int groups = A.tile * V / A.cg;
    Held<T, V, POOL, R> H;
    Pack<T, V> D[R];
    H.load_all(A, P, x);
    const int64_t yrow = (int64_t)P.sample * A.total + P.r0 + P.lane;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < P.left) D[i] = load<T, V>(dy + (yrow + (int64_t)i * P.lanes) * A.yp + P.c0);
    float a[V], m[V], be[V], rs[V], db[V], dg[V];
    if (P.left) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int64_t g = (int64_t)P.sample * A.groups + A.gdiv.div(P.c0 + e);
            m[e] = mean[g];
            rs[e] = rstd[g];
            a[e] = (gamma ? gamma[P.c0 + e] : 1.f) * rs[e];
            be[e] = beta ? beta[P.c0 + e] : 0.f;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) db[e] = dg[e] = 0.f;
    auto grad = [&](float (&f)[V], float (&g)[V]) {  // f: x - mean, g: du
        float u[V];
        vsub<V>(f, f, m);
        vfma<V>(u, a, f, be);
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] *= act_grad<T, ACT>(u[e], A.slope);
    };
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < P.left) {
            float f[V], g[V], d[V];
            unpack<T, V>(D[i], d);
            if (POOL == CF_POOL_AVG) {
#pragma unroll
                for (int j = 0; j < H.K; ++j) {
                    unpack<T, V>(H.t[i][j], f);
#pragma unroll
                    for (int e = 0; e < V; ++e) g[e] = 0.125f * d[e];
                    grad(f, g);
                    vadd<V>(db, db, g);
                    vfma<V>(dg, g, f, dg);
                }
            } else {
                if constexpr (POOL == CF_POOL_MAX)
                    window_max<T, V>(H.t[i], a, f);
                else
                    unpack<T, V>(H.t[i][0], f);
                grad(f, d);
                vadd<V>(db, db, d);
                vfma<V>(dg, d, f, dg);
            }
        }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        sb[e * kSmallThreads + threadIdx.x] = db[e];
        sg[e * kSmallThreads + threadIdx.x] = P.left ? dg[e] * rs[e] : 0.f;
    }
    __syncthreads();
    // a channel's row lanes are added up by as many neighbouring threads as the block has for it; its sums go to slot 0
    const int wide = A.tile * V, cb = blockIdx.y * wide;
    int lp = 1;
    while (2 * lp <= 32 && 2 * lp <= P.lanes && 2 * lp * wide <= kSmallThreads) lp *= 2;
    float2 sums[V > 1 ? V : 1];  // of the channels this thread takes, in turn: wide <= kSmallThreads V
    int mine = 0;
    for (int i = threadIdx.x / lp; i < (wide + 31) / 32 * 32; i += kSmallThreads / lp, ++mine) {
        float tb = 0.f, tg = 0.f;
        if (i < wide)
            for (int l = threadIdx.x & (lp - 1); l < P.lanes; l += lp) {
                tb += sb[i % V * kSmallThreads + l * A.tile + i / V];
                tg += sg[i % V * kSmallThreads + l * A.tile + i / V];
            }
        for (int o = lp / 2; o; o >>= 1) {
            tb += __shfl_xor_sync(~0u, tb, o);
            tg += __shfl_xor_sync(~0u, tg, o);
        }
#pragma unroll
        for (int w = 0; w < V; ++w)
            if (w == mine) sums[w] = make_float2(tb, tg);
    }
    __syncthreads();
    mine = 0;
    for (int i = threadIdx.x / lp; i < (wide + 31) / 32 * 32; i += kSmallThreads / lp, ++mine)
        if (i < wide && (threadIdx.x & (lp - 1)) == 0) {
            float2 t = sums[0];
#pragma unroll
            for (int w = 1; w < V; ++w)
                if (w == mine) t = sums[w];
            A.part[((int64_t)P.sample * A.chunks + P.rank) * A.c + cb + i] = t;
            const float ga = gamma ? gamma[cb + i] : 1.f;
            sb[i] = t.x * ga;
            sg[i] = t.y * ga;
        }
    if (dx == nullptr) return;
    __syncthreads();
    cluster_begun();
    for (int g = threadIdx.x >> 5; g < groups; g += kSmallWarps) {
        float s1 = 0.f, s2 = 0.f;
        for (int i = threadIdx.x & 31; i < A.cg; i += 32) {
            s1 += sb[g * A.cg + i];
            s2 += sg[g * A.cg + i];
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if ((threadIdx.x & 31) < A.chunks) store_remote(&ex[P.rank * groups + g], threadIdx.x & 31, make_float2(s1, s2));
    }
    cluster_sync();
    float2* stat = ex + A.chunks * groups;
    for (int g = threadIdx.x; g < groups; g += kSmallThreads) {
        float s1 = 0.f, s2 = 0.f;
        for (int r = 0; r < A.chunks; ++r) {
            s1 += ex[r * groups + g].x;
            s2 += ex[r * groups + g].y;
        }
        const float inv = 1.f / ((float)A.s * (float)A.cg);
        stat[g] = make_float2(s1 * inv, s2 * inv);
    }
    __syncthreads();
    if (!P.left) return;
    float k0[V], k1[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float2 t = stat[A.gdiv.div(P.col * V + e)];
        k0[e] = -rs[e] * t.x;
        k1[e] = -rs[e] * rs[e] * t.y;
    }
    const Window W(A);
    T* os = dx + (int64_t)P.sample * A.s * A.xp + P.c0;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < P.left) {
            const int64_t row = P.r0 + P.lane + i * P.lanes;
            T* o = os + (H.K == 1 ? row * A.xp : window_at(A, row));
            float f[V], g[V], d[V], lin[V];
            unpack<T, V>(D[i], d);
            if constexpr (POOL == CF_POOL_NONE) {
                unpack<T, V>(H.t[i][0], f);
                grad(f, d);
                vfma<V>(lin, k1, f, k0);
                vfma<V>(lin, a, d, lin);
                store<T, V>(o, lin);
            } else {
                float best[V];
                if (POOL == CF_POOL_MAX) {
                    window_max<T, V>(H.t[i], a, best);
#pragma unroll
                    for (int e = 0; e < V; ++e) f[e] = best[e];
                    grad(f, d);
#pragma unroll
                    for (int e = 0; e < V; ++e) d[e] *= a[e];
                }
#pragma unroll
                for (int j = 0; j < H.K; ++j) {
                    unpack<T, V>(H.t[i][j], f);
                    if (POOL == CF_POOL_MAX) {
                        float c[V];
                        vsub<V>(c, f, m);
                        vfma<V>(lin, k1, c, k0);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const bool hit = f[e] == best[e];
                            lin[e] += hit ? d[e] : 0.f;
                            d[e] = hit ? 0.f : d[e];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < V; ++e) g[e] = 0.125f * d[e];
                        grad(f, g);
                        vfma<V>(lin, k1, f, k0);
                        vfma<V>(lin, a, g, lin);
                    }
                    store<T, V>(o + W.at(j), lin);
                }
            }
        }
}

// dbeta and dgamma from `rows` rows of channel sums: 32 channels a block, a row lane to each warp.
__global__ void __launch_bounds__(kThreads) gn_channels_kernel(const float2* part, int64_t rows, int c, float* dgamma,
                                                              float* dbeta) {
    __shared__ float2 red[kWarps][33];
    grid_wait();
    const int ch = blockIdx.x * 32 + (threadIdx.x & 31), l = threadIdx.x >> 5;
    float tb = 0.f, tg = 0.f;
    if (ch < c) {
#pragma unroll 4
        for (int64_t i = l; i < rows; i += kWarps) {
            const float2 v = part[i * c + ch];
            tb += v.x;
            tg += v.y;
        }
    }
    red[l][threadIdx.x & 31] = make_float2(tb, tg);
    __syncthreads();
    if (l == 0 && ch < c) {
        for (int i = 1; i < kWarps; ++i) {
            tb += red[i][threadIdx.x].x;
            tg += red[i][threadIdx.x].y;
        }
        if (dbeta) dbeta[ch] = tb;
        if (dgamma) dgamma[ch] = tg;
    }
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
    // window_at divides a window's number in 32 bits
    if (d->pool != CF_POOL_NONE && d->d / 2 * (d->h / 2) * (d->w / 2) > (int64_t)UINT32_MAX) return CF_ERR_UNSUPPORTED;
    return CF_OK;
}

// Values of a vector access: 16 bytes where channels and pitches allow it, else four values, in bf16 two, else one.
// (bf16 in twos against one by one: 2 x 82 95 76 x 58 forward 86 : 103 us, 5 x 89 81 95 x 26 of 90 backward 370 : 409.)
int vec_of(const cf_gn_desc* d) {
    const int64_t xp = d->x_pitch ? d->x_pitch : d->c, yp = d->y_pitch ? d->y_pitch : d->c;
    for (int v = d->dtype == CF_DT_F32 ? 4 : 8; v >= (d->dtype == CF_DT_F32 ? 4 : 2); v /= 2)
        if (d->c % v == 0 && xp % v == 0 && yp % v == 0) return v;
    return 1;
}
// Chunks are cut for the blocks that fit 152 SMs at once, whatever the device: the workspace's size and the sums' order depend
// on the descriptor alone.
int plan_blocks(const cf_gn_desc* d, bool backward) { return 152 * (backward ? 2 : 3); }
// Voxels of a thread in a chunk, at most (8 x 128^3 x 32 forward: 329 us; with 32 336, with 16 372, with 256 333; 8 x 64^3 x 64
// backward 153, 155, 188, 158).
constexpr int kMostRows = 64;

GnArgs make_args(const cf_gn_desc* d, bool backward) {
    GnArgs A{};
    const int v = vec_of(d);
    A.n = (int)d->n, A.d = (int)d->d, A.h = (int)d->h, A.w = (int)d->w, A.s = d->d * d->h * d->w;
    A.c = d->c, A.groups = d->groups, A.cg = d->c / d->groups;
    A.xp = d->x_pitch ? d->x_pitch : d->c, A.yp = d->y_pitch ? d->y_pitch : d->c;
    A.slope = d->slope, A.eps = d->eps;
    const int vc = d->c / v;
    A.tiles = (vc + kThreads - 1) / kThreads;
    A.tile = (vc + A.tiles - 1) / A.tiles;
    const int win = d->pool != CF_POOL_NONE ? 8 : 1;
    A.total = A.s / win;
    if (win == 8) A.w2 = FastDiv::make((uint32_t)(d->w / 2)), A.h2 = FastDiv::make((uint32_t)(d->h / 2));
    // items (voxels, or windows of eight) of a row lane in a chunk: an even share of as many waves of blocks as it takes for
    // no more than kMostRows voxels, but four (a window) at least
    const int64_t lanes = kThreads / A.tile, blocks = lanes * plan_blocks(d, backward);
    const int64_t share = (A.total * A.n * A.tiles + blocks - 1) / blocks, waves = (share * win + kMostRows - 1) / kMostRows;
    const int64_t per = std::max<int64_t>(win == 8 ? 1 : 4, (share + waves - 1) / waves);
    A.rows = (int)std::min(A.total, lanes * per);
    A.srows = win * A.rows;
    A.chunks = (int)std::min<int64_t>((A.total + A.rows - 1) / A.rows, INT32_MAX);
    A.tdiv = FastDiv::make((uint32_t)A.tile);
    A.cdiv = FastDiv::make((uint32_t)A.chunks);
    A.gdiv = FastDiv::make((uint32_t)A.cg);
    return A;
}

// Whether the blocks of every launch and the rows of statistics can be counted in 32 bits (what fits the device's memory can).
bool counts_ok(const GnArgs& A) {
    const int64_t most = INT32_MAX, n = A.n;
    return n * A.chunks + A.c / kThreads + 1 <= most && n * A.groups <= most && (int64_t)A.chunks * A.tiles <= most &&
           n * A.c / kThreads + 1 <= most && A.tiles <= 65535;
}

// Items (vectors, or windows of eight) that a thread of the small kernels holds.
constexpr int kSmallItems = 16, kSmallWindows = 2;
constexpr int kMaxCluster = 16;
// Bytes of x up to which a call goes to the small kernels where they take its shape.
constexpr int64_t kSmallBytes = 16 << 20;

// The small kernels' way to take a call: columns of whole groups, and the blocks of a cluster; false where the sample does not
// fit.  Sets tile, tiles, chunks (the cluster's blocks) and rows (of a block).
bool small_args(const cf_gn_desc* d, bool backward, GnArgs& A) {
    const int v = vec_of(d), win = d->pool != CF_POOL_NONE ? 8 : 1, vc = d->c / v;
    const int64_t size = d->dtype == CF_DT_F32 ? 4 : 2;
    if (A.s * A.n * A.c > kSmallBytes / size) return false;
    int a = A.cg, b = v;
    while (b) {
        const int t = a % b;
        a = b, b = t;
    }
    const int least = A.cg / a;  // vectors that are whole groups: lcm(cg, v) / v
    const int most = win == 8 ? kSmallWindows : backward ? kSmallItems / 2 : kSmallItems;
    // of all ways to cut the columns and the rows, the one whose waves of blocks take the fewest steps: a block's start, its
    // items one after the other, and the exchange where a sample has several blocks
    int64_t best = INT64_MAX;
    for (int split = 1; split <= vc / least; ++split) {
        const int tile = vc / split;
        if (split > 1 && (int64_t)tile * v * size < 64) break;
        if ((vc / least) % split || tile > kSmallThreads || tile * v / A.cg > 64) continue;
        const int64_t lanes = kSmallThreads / tile;
        for (int q = 1; q <= kMaxCluster; q *= 2) {
            const int64_t rows = (A.total + q - 1) / q, items = (rows + lanes - 1) / lanes;
            if (items > most) continue;
            const int64_t waves = (A.n * (int64_t)split * q + 2 * 152 - 1) / (2 * 152);
            const int64_t cost = waves * (6 + items * (win == 8 ? 4 : 1) + (q > 1 ? 4 : 0));
            if (cost < best) {
                best = cost;
                A.tile = tile, A.tiles = split, A.chunks = q;
                A.rows = (int)rows;
            }
            if (items == 1) break;
        }
    }
    if (best == INT64_MAX) return false;
    A.tdiv = FastDiv::make((uint32_t)A.tile);
    return true;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Places the workspace at `base` (NULL: to count) and returns its size.
size_t place(GnArgs& A, bool backward, bool small, char* base) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = base + at;
        at += up256(bytes);
        return p;
    };
    const size_t chunks = (size_t)A.n * A.chunks, nc = (size_t)A.n * A.c;
    if (small) {
        if (backward) A.part = reinterpret_cast<float2*>(take(chunks * A.c * sizeof(float2)));
        return std::max<size_t>(at, 256);
    }
    A.part = reinterpret_cast<float2*>(take(chunks * (backward ? (size_t)A.c : (size_t)A.tiles * A.groups) * sizeof(float2)));
    A.coef = reinterpret_cast<float4*>(take(nc * sizeof(float4)));
    if (backward) {
        A.lin = reinterpret_cast<float2*>(take(nc * sizeof(float2)));
        A.chan = reinterpret_cast<float2*>(take(nc * sizeof(float2)));
    }
    return at;
}

// A launch that may begin before the one before it in the stream has ended (its kernel calls grid_wait).
template <typename K, typename... P>
void launch_after(const LaunchCtx& ctx, dim3 grid, int shared, K kern, P... args) {
    if (shared > (48 << 10)) cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int V, int POOL, int ACT>
void launch_fwd(const LaunchCtx& ctx, const GnArgs& A, const void* x, const float* gamma, const float* beta, void* y, float* mean,
                float* rstd) {
    const dim3 grid((unsigned)(A.n * A.chunks), A.tiles);
    gn_stats_kernel<T, V><<<grid, kThreads, 0, ctx.stream>>>(A, static_cast<const T*>(x));
    launch_after(ctx, dim3(A.n * A.groups), 0, gn_finish_kernel<V>, A, gamma, beta, mean, rstd);
    launch_after(ctx, grid, 0, gn_apply_kernel<T, V, POOL, ACT>, A, static_cast<const T*>(x), static_cast<T*>(y));
}

template <typename T, int V, int POOL, int ACT>
void launch_bwd(const LaunchCtx& ctx, const GnArgs& A, const void* x, const float* gamma, const float* beta, const float* mean,
                const float* rstd, const void* dy, void* dx, float* dgamma, float* dbeta) {
    const T *xt = static_cast<const T*>(x), *dyt = static_cast<const T*>(dy);
    const int work = A.n * A.chunks, blocks = dx ? work : 0, more = dgamma || dbeta ? (A.c + kThreads - 1) / kThreads : 0;
    gn_coef_kernel<<<(unsigned)(((int64_t)A.n * A.c + kThreads - 1) / kThreads), kThreads, 0, ctx.stream>>>(A, gamma, beta, mean, rstd);
    constexpr int kRing = Rows<T, V, POOL != CF_POOL_NONE>::kBytes, kSums = 2 * kThreads * V * (int)sizeof(float);
    launch_after(ctx, dim3(work, A.tiles), std::max(kRing, kSums), gn_bwd_sums_kernel<T, V, POOL, ACT>, A, xt, dyt);
    launch_after(ctx, dim3(A.n * A.groups), 0, gn_bwd_finish_kernel, A, gamma);
    if (blocks + more > 0)
        launch_after(ctx, dim3(blocks + more, A.tiles), kRing, gn_bwd_apply_kernel<T, V, POOL, ACT>, A, xt, dyt, static_cast<T*>(dx),
                     blocks, dgamma, dbeta);
}

// A launch in clusters of A.chunks blocks.
template <typename K, typename... P>
cudaError_t launch_small(const LaunchCtx& ctx, const GnArgs& A, int groups, K kern, P... args) {
    const size_t sm = (size_t)(A.chunks + 1) * groups * sizeof(float2);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(A.n * A.chunks), (unsigned)A.tiles);
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = sm;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)A.chunks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (A.chunks > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int V, int POOL, int ACT>
void launch_small_fwd(const LaunchCtx& ctx, const GnArgs& A, const void* x, const float* gamma, const float* beta, void* y, float* mean,
                      float* rstd) {
    const int lanes = kSmallThreads / A.tile, items = (A.rows + lanes - 1) / lanes, groups = A.tile * V / A.cg;
    const T* xt = static_cast<const T*>(x);
    T* yt = static_cast<T*>(y);
    constexpr int kMost = POOL == CF_POOL_NONE ? kSmallItems : kSmallWindows, kFew = POOL == CF_POOL_NONE ? kSmallItems / 4 : 1;
    if (items <= kFew)
        launch_small(ctx, A, groups, gn_small_fwd_kernel<T, V, POOL, ACT, kFew>, A, xt, gamma, beta, yt, mean, rstd);
    else
        launch_small(ctx, A, groups, gn_small_fwd_kernel<T, V, POOL, ACT, kMost>, A, xt, gamma, beta, yt, mean, rstd);
}

template <typename T, int V, int POOL, int ACT>
void launch_small_bwd(const LaunchCtx& ctx, const GnArgs& A, const void* x, const float* gamma, const float* beta, const float* mean,
                      const float* rstd, const void* dy, void* dx, float* dgamma, float* dbeta) {
    const int lanes = kSmallThreads / A.tile, items = (A.rows + lanes - 1) / lanes, groups = A.tile * V / A.cg;
    const T *xt = static_cast<const T*>(x), *dyt = static_cast<const T*>(dy);
    T* dxt = static_cast<T*>(dx);
    constexpr int kMost = POOL == CF_POOL_NONE ? kSmallItems / 2 : kSmallWindows, kFew = POOL == CF_POOL_NONE ? kSmallItems / 8 : 1;
    if (items <= kFew)
        launch_small(ctx, A, groups, gn_small_bwd_kernel<T, V, POOL, ACT, kFew>, A, xt, gamma, beta, mean, rstd, dyt, dxt);
    else
        launch_small(ctx, A, groups, gn_small_bwd_kernel<T, V, POOL, ACT, kMost>, A, xt, gamma, beta, mean, rstd, dyt, dxt);
    if (dgamma || dbeta)
        launch_after(ctx, dim3((A.c + 31) / 32), 0, gn_channels_kernel, (const float2*)A.part, (int64_t)A.n * A.chunks, A.c, dgamma, dbeta);
}

// Calls f<T, V, POOL, ACT>(...) for the descriptor.
#define CF_GN_ACT(d, f, T, V, POOL, ...) \
    ((d)->act == CF_ACT_SILU ? f<T, V, POOL, CF_ACT_SILU>(__VA_ARGS__) : f<T, V, POOL, CF_ACT_LRELU>(__VA_ARGS__))
#define CF_GN_POOL(d, f, V, ...)                                           \
    do {                                                                   \
        if ((d)->pool == CF_POOL_NONE)                                     \
            CF_GN_ACT(d, f, uint16_t, V, CF_POOL_NONE, __VA_ARGS__);       \
        else if ((d)->pool == CF_POOL_MAX)                                 \
            f<uint16_t, V, CF_POOL_MAX, CF_ACT_LRELU>(__VA_ARGS__);        \
        else                                                               \
            CF_GN_ACT(d, f, uint16_t, V, CF_POOL_AVG, __VA_ARGS__);        \
    } while (0)
#define CF_GN_DISPATCH(d, f, ...)                                          \
    do {                                                                   \
        const int vec = vec_of(d);                                         \
        if ((d)->dtype == CF_DT_F32) {                                     \
            if (vec > 1)                                                   \
                CF_GN_ACT(d, f, float, 4, CF_POOL_NONE, __VA_ARGS__);      \
            else                                                           \
                CF_GN_ACT(d, f, float, 1, CF_POOL_NONE, __VA_ARGS__);      \
        } else if (vec == 8) {                                             \
            CF_GN_POOL(d, f, 8, __VA_ARGS__);                              \
        } else if (vec == 4) {                                             \
            CF_GN_POOL(d, f, 4, __VA_ARGS__);                              \
        } else if (vec == 2) {                                             \
            CF_GN_POOL(d, f, 2, __VA_ARGS__);                              \
        } else {                                                           \
            CF_GN_POOL(d, f, 1, __VA_ARGS__);                              \
        }                                                                  \
    } while (0)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace cf

using namespace cf;

extern "C" {

size_t cf_group_norm_workspace_size(const cf_gn_desc* desc, int32_t backward) {
    if (!desc_ok(desc) || supported(desc) != CF_OK) return 0;
    GnArgs A = make_args(desc, backward != 0);
    if (!counts_ok(A)) return 0;
    const bool small = small_args(desc, backward != 0, A);
    return place(A, backward != 0, small, nullptr);
}

cf_status cf_group_norm_fwd(const cf_gn_desc* desc, const void* x, const float* gamma, const float* beta, void* y,
                            float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream) {
    if (!desc_ok(desc) || x == nullptr || y == nullptr) return CF_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) || !aligned16(rstd) ||
        !aligned16(ws))
        return CF_ERR_INVALID_ARG;
    if (const cf_status st = supported(desc); st != CF_OK) return st;
    GnArgs A = make_args(desc, false);
    if (!counts_ok(A)) return CF_ERR_UNSUPPORTED;
    const bool small = small_args(desc, false, A);
    if (ws == nullptr || ws_bytes < place(A, false, small, nullptr)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    place(A, false, small, static_cast<char*>(ws));
    if (small)
        CF_GN_DISPATCH(desc, launch_small_fwd, ctx, A, x, gamma, beta, y, mean, rstd);
    else
        CF_GN_DISPATCH(desc, launch_fwd, ctx, A, x, gamma, beta, y, mean, rstd);
    return cudaGetLastError() == cudaSuccess ? CF_OK : CF_ERR_CUDA;
}

cf_status cf_group_norm_bwd(const cf_gn_desc* desc, const void* x, const float* gamma, const float* beta,
                            const float* mean, const float* rstd, const void* dy, void* dx, float* dgamma,
                            float* dbeta, void* ws, size_t ws_bytes, void* stream) {
    if (!desc_ok(desc) || x == nullptr || mean == nullptr || rstd == nullptr || dy == nullptr) return CF_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(dy) || !aligned16(dx) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) ||
        !aligned16(rstd) || !aligned16(dgamma) || !aligned16(dbeta) || !aligned16(ws))
        return CF_ERR_INVALID_ARG;
    if (const cf_status st = supported(desc); st != CF_OK) return st;
    GnArgs A = make_args(desc, true);
    if (!counts_ok(A)) return CF_ERR_UNSUPPORTED;
    const bool small = small_args(desc, true, A);
    if (ws == nullptr || ws_bytes < place(A, true, small, nullptr)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    place(A, true, small, static_cast<char*>(ws));
    if (small)
        CF_GN_DISPATCH(desc, launch_small_bwd, ctx, A, x, gamma, beta, mean, rstd, dy, dx, dgamma, dbeta);
    else
        CF_GN_DISPATCH(desc, launch_bwd, ctx, A, x, gamma, beta, mean, rstd, dy, dx, dgamma, dbeta);
    return cudaGetLastError() == cudaSuccess ? CF_OK : CF_ERR_CUDA;
}

}  // extern "C"
