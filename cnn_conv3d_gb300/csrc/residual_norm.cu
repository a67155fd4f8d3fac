// residual_norm.cu -- the norms before and after a block with the gated, scaled sum between (r = x + scale gate N_post(f),
// h = N_pre(r)), forward and backward, with their entry points.
//
// Backward, per row, with vh the normalised values, u = gamma_pre dh and dv = scale gate gamma_post dx:
//   dx = dr + rstd_r (u - mean u - rh mean(u rh))        (the mean of u for the layer norm only)
//   df = rstd_f (dv - mean dv - fh mean(dv fh))
// and four sums over rows are enough for all five vectors' gradients: A = sum dx fh, B = sum dx, C = sum dh rh, D = sum dh give
//   dgate = scale (gamma_post A + beta_post B),  dgamma_post = scale gate A,  dbeta_post = scale gate B,  dgamma_pre = C,
//   dbeta_pre = D                                 (gate's factor inside the sum over the samples where each has its own)
//
// Every tensor is read and written once, so memory is the bound, and what keeps from it is the latency of the rows' sums.  A row is held
// by as many threads as give each eight of its values: part of a warp up to 256 values, a block up to 4096; longer rows are read again
// for each sum.  Columns' sums stay in registers over a block's rows, whose chunks depend on the sizes alone: results do not change
// from run to run.  bf16 RMS norms of 67M values, cold (8 us of it measuring), forward and backward: rows of 256 values 95 and 153 us
// (5.6 and 5.3 TB/s), of 1024 107 and 198 us (5.0 and 4.1), of 4096 119 and 216 us (4.5 and 3.7), of 8192 178 and 400 us (3.0 and 2.0).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "cf_internal.h"
#include "cf_ptx.cuh"
#include "cf_two.cuh"

namespace cf {
namespace {

struct RnArgs {
    int64_t rows, per;         // per: rows of a sample
    int c, post, pre;
    int gate_each, pre_each;   // a vector for each sample
    float eps, scale, inv_c;
    int samples, chunks;       // chunks of a sample's rows, `chunk` rows each
    int64_t chunk;
    const float *post_gamma, *post_beta, *gate, *pre_gamma, *pre_beta;
};

__device__ __forceinline__ void store(uint16_t* p, int64_t i, float v) { p[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ float at_or(const float* p, int64_t i, float other) { return p ? p[i] : other; }

constexpr int kThreads = 256;

// Sums over the block, the same in every thread.
__device__ __forceinline__ float2 block_sum(float a, float b, float2* red) {
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(~0u, a, o);
        b += __shfl_xor_sync(~0u, b, o);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) a += red[i].x, b += red[i].y;
    return make_float2(a, b);
}

// ------------------------------------------------------------------------------------------------ rows that registers hold at once
// Eight values of a row to a thread: T threads of a warp to a row of up to 256 values (T a power of two, 32 / T rows of a warp at
// once), or all of a block's (WIDE, up to 4096).  Where c is a multiple of eight a thread has neighbouring columns in 16-byte
// accesses, otherwise columns T apart.  A block has the rows of a chunk of one sample, keeps the vectors in registers over them and
// fetches a row's values while the one before is worked on.
constexpr int kMostWide = 4096;

template <bool VEC>
struct Cols {
    static constexpr bool vec = VEC;
    int t, T, c;
    __device__ __forceinline__ int at(int e) const { return vec ? 8 * t + e : t + T * e; }
    __device__ __forceinline__ bool has(int e) const { return vec ? 8 * t < c : t + T * e < c; }
};

template <typename S>
struct Raw {  // eight values as they are stored
    uint32_t u[sizeof(S) * 2];
};
template <typename C_>
__device__ __forceinline__ Raw<uint16_t> load8(const uint16_t* p, int64_t o, const C_& C) {
    Raw<uint16_t> r;
    if (C.vec) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (C.has(0)) v = __ldcg(reinterpret_cast<const uint4*>(p + o + 8 * C.t));
        r.u[0] = v.x, r.u[1] = v.y, r.u[2] = v.z, r.u[3] = v.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t a = C.has(2 * e) ? p[o + C.at(2 * e)] : 0, b = C.has(2 * e + 1) ? p[o + C.at(2 * e + 1)] : 0;
            r.u[e] = a | b << 16;
        }
    }
    return r;
}
template <typename C_>
__device__ __forceinline__ Raw<float> load8(const float* p, int64_t o, const C_& C) {
    Raw<float> r;
    if (C.vec) {
        uint4 v = make_uint4(0, 0, 0, 0), w = v;
        if (C.has(0)) {
            const uint4* q = reinterpret_cast<const uint4*>(p + o + 8 * C.t);
            v = __ldcg(q), w = __ldcg(q + 1);
        }
        r.u[0] = v.x, r.u[1] = v.y, r.u[2] = v.z, r.u[3] = v.w, r.u[4] = w.x, r.u[5] = w.y, r.u[6] = w.z, r.u[7] = w.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.u[e] = C.has(e) ? __float_as_uint(p[o + C.at(e)]) : 0;
    }
    return r;
}
// As four pairs, with which all arithmetic is done.
__device__ __forceinline__ void unpack(const Raw<uint16_t>& r, uint64_t (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = two(__uint_as_float(r.u[e] << 16), __uint_as_float(r.u[e] & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const Raw<float>& r, uint64_t (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = two(__uint_as_float(r.u[2 * e]), __uint_as_float(r.u[2 * e + 1]));
}
__device__ __forceinline__ void spread(const uint64_t (&p)[4], float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) apart(p[e], v[2 * e], v[2 * e + 1]);
}
template <typename C_>
__device__ __forceinline__ void store8(uint16_t* p, int64_t o, const C_& C, const uint64_t (&q)[4]) {
    float v[8];
    spread(q, v);
    if (C.vec) {
        if (C.has(0))
            *reinterpret_cast<uint4*>(p + o + 8 * C.t) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (C.has(e)) store(p, o + C.at(e), v[e]);
    }
}
template <typename C_>
__device__ __forceinline__ void store8(float* p, int64_t o, const C_& C, const uint64_t (&q)[4]) {
    float v[8];
    spread(q, v);
    if (C.vec) {
        if (C.has(0)) {
            float4* to = reinterpret_cast<float4*>(p + o + 8 * C.t);
            to[0] = make_float4(v[0], v[1], v[2], v[3]), to[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (C.has(e)) p[o + C.at(e)] = v[e];
    }
}
// A vector's eight values, `other` where there is no vector, and 0 in columns that the thread does not have: what it makes of those
// adds nothing to a row's sums.
template <typename C_>
__device__ __forceinline__ void vector8(const float* p, int64_t o, const C_& C, float other, uint64_t (&q)[4]) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = C.has(e) ? other : 0.f;
    if (p != nullptr) {
        if (C.vec) {
            if (C.has(0)) {
                const float4* from = reinterpret_cast<const float4*>(p + o + 8 * C.t);
                const float4 a = from[0], b = from[1];
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (C.has(e)) v[e] = p[o + C.at(e)];
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = two(v[2 * e], v[2 * e + 1]);
}

// Sums over the threads of B rows, the same in each of them.  WIDE: one barrier of the rows' T threads, the buffers in turn; it also
// tells all of them of a thread that has failed.
constexpr int kMostRows = 2;
template <bool WIDE>
struct RowSum {
    float (*red)[16][2 * kMostRows];
    int turn = 0, T;
    int failed = 0;
    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N]) {
        for (int o = (WIDE ? 32 : T) >> 1; o; o >>= 1)
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] += __shfl_xor_sync(~0u, v[e], o);
        if (WIDE) {
            float(*r)[2 * kMostRows] = red[turn];
            turn ^= 1;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int e = 0; e < N; ++e) r[threadIdx.x >> 5][e] = v[e];
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.s32 p, %0, 0;\n\t"
                "barrier.cta.red.or.pred q, 1, %1, p;\n\t"
                "selp.s32 %0, 1, 0, q;\n\t}\n"
                : "+r"(failed)
                : "r"(T)
                : "memory");
            // up to 16 warps' sums: a lane to each
            const int lane = threadIdx.x & 31;
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = lane < T >> 5 ? r[lane][e] : 0.f;
            for (int o = T > 256 ? 8 : T > 128 ? 4 : T > 64 ? 2 : 1; o; o >>= 1)
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] += __shfl_xor_sync(~0u, v[e], o);
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = __shfl_sync(~0u, v[e], 0);
        }
    }
};

// (mean, 1 / width) of B rows that their threads hold eight values of each (0 in columns that they do not have).
template <bool WIDE, int B, typename C_>
__device__ __forceinline__ void stats8(const RnArgs& A, int kind, const C_& C, RowSum<WIDE>& sum, const uint64_t (&v)[B][4], float2 (&st)[B]) {
#pragma unroll
    for (int k = 0; k < B; ++k) st[k] = make_float2(0.f, 1.f);
    if (kind == CF_NORM_NONE) return;
    float s[B];
    if (kind == CF_NORM_LAYER) {
#pragma unroll
        for (int k = 0; k < B; ++k) s[k] = total(add2(add2(v[k][0], v[k][1]), add2(v[k][2], v[k][3])));
        sum(s);
#pragma unroll
        for (int k = 0; k < B; ++k) st[k].x = s[k] * A.inv_c;
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
        uint64_t q = 0;
        const uint64_t less = both(-st[k].x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint64_t t = add2(v[k][e], less);
            if (!C.vec) {
                float a, b;
                apart(t, a, b);
                t = two(C.has(2 * e) ? a : 0.f, C.has(2 * e + 1) ? b : 0.f);
            }
            q = fma2(t, t, q);
        }
        s[k] = C.vec && !C.has(0) ? 0.f : total(q);
    }
    sum(s);
#pragma unroll
    for (int k = 0; k < B; ++k) st[k].y = rsqrtf(s[k] * A.inv_c + A.eps);
}

// A block's chunk of rows, and the thread's place in them.
struct Place {
    int64_t from, to, sample;
    int step;  // rows at once
};
template <bool WIDE, typename C_>
__device__ __forceinline__ Place place_of(const RnArgs& A, int T, C_& C) {
    Place P;
    C.c = A.c, C.T = T;
    C.t = WIDE ? threadIdx.x : threadIdx.x & (T - 1);
    P.sample = blockIdx.x / A.chunks;
    const int64_t first = P.sample * A.per + (blockIdx.x - P.sample * A.chunks) * A.chunk;
    P.to = min(min(first + A.chunk, (P.sample + 1) * A.per), A.rows);
    P.step = WIDE ? 1 : kThreads / T;
    P.from = first + (WIDE ? 0 : (int)threadIdx.x / T);
    return P;
}

// The vectors of a thread's columns: p = a fh + b, h = g rh + beta.
struct FwdVectors {
    uint64_t a[4], b[4], g[4], beta[4];
    template <typename C_>
    __device__ __forceinline__ FwdVectors(const RnArgs& A, const C_& C, int64_t sample) {
        uint64_t gate[4];
        vector8(A.gate, A.gate_each ? sample * A.c : 0, C, 1.f, gate);
        vector8(A.post_gamma, 0, C, 1.f, a);
        vector8(A.post_beta, 0, C, 0.f, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t s = mul2(both(A.scale), gate[e]);
            a[e] = mul2(a[e], s), b[e] = mul2(b[e], s);
        }
        vector8(A.pre_gamma, A.pre_each ? sample * A.c : 0, C, 1.f, g);
        vector8(A.pre_beta, A.pre_each ? sample * A.c : 0, C, 0.f, beta);
    }
};
// B rows, `step` apart from row i on, from their values v of x and w of f (0 where the thread has none).
template <typename S, typename F, bool WIDE, int B, typename C_>
__device__ __forceinline__ void fwd_rows(const RnArgs& A, const C_& C, RowSum<WIDE>& sum, const FwdVectors& V, bool with_f, int64_t i, int step,
                                         const bool (&mine)[B], uint64_t (&v)[B][4], uint64_t (&w)[B][4], S* r, F* h, float4* stats) {
    float2 sf[B], sr[B];
#pragma unroll
    for (int k = 0; k < B; ++k) sf[k] = make_float2(0.f, 1.f);
    if (with_f) {
        stats8<WIDE>(A, A.post, C, sum, w, sf);
#pragma unroll
        for (int k = 0; k < B; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[k][e] = add2(v[k][e], fma2(V.a[e], mul2(add2(w[k][e], both(-sf[k].x)), both(sf[k].y)), V.b[e]));
    }
#pragma unroll
    for (int k = 0; k < B; ++k)
        if (r && mine[k]) store8(r, (i + k * step) * A.c, C, v[k]);
    stats8<WIDE>(A, A.pre, C, sum, v, sr);
#pragma unroll
    for (int k = 0; k < B; ++k) {
        if (h && mine[k]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[k][e] = fma2(mul2(add2(v[k][e], both(-sr[k].x)), both(sr[k].y)), V.g[e], V.beta[e]);
            store8(h, (i + k * step) * A.c, C, v[k]);
        }
        if (stats && mine[k] && C.t == 0) stats[i + k * step] = make_float4(sf[k].x, sf[k].y, sr[k].x, sr[k].y);
    }
}

template <typename S, typename F, bool WIDE, bool VEC>
__global__ void __launch_bounds__(WIDE ? kMostWide / 8 : kThreads, WIDE ? 1 : 3) rn_fwd_kernel(const RnArgs A, int T, const S* x, const F* f, S* r,
                                                                                              F* h, float4* stats) {
    __shared__ float red[2][16][2 * kMostRows];
    Cols<VEC> C;
    const Place P = place_of<WIDE>(A, T, C);
    RowSum<WIDE> sum{red, 0, T};
    const FwdVectors V(A, C, P.sample);
    // all threads of a warp go round as often, for the shuffles
    const int64_t rounds = (P.to - (P.from - (WIDE ? 0 : (int)threadIdx.x / T)) + P.step - 1) / P.step;
    Raw<S> xn{};
    Raw<F> fn{};
    if (P.from < P.to) {
        xn = load8(x, P.from * A.c, C);
        if (f) fn = load8(f, P.from * A.c, C);
    }
    for (int64_t k = 0; k < rounds; ++k) {
        const int64_t i = P.from + k * P.step;
        uint64_t v[1][4], w[1][4];
        unpack(xn, v[0]);
        unpack(fn, w[0]);
        if (i + P.step < P.to) {
            xn = load8(x, (i + P.step) * A.c, C);
            if (f) fn = load8(f, (i + P.step) * A.c, C);
        }
        const bool mine[1] = {i < P.to};
        fwd_rows(A, C, sum, V, f != nullptr, i, 0, mine, v, w, r, h, stats);
    }
}

// Backward: dv = a dx, u = g dh, and the sums over the thread's rows.  In columns that a thread does not have a and g are 0, so that
// what it makes there of the means adds nothing to a row's sums (its own, of those columns, go nowhere).
struct BwdVectors {
    uint64_t a[4], g[4], sa[4] = {}, sb[4] = {}, sc[4] = {}, sd[4] = {};
    template <typename C_>
    __device__ __forceinline__ BwdVectors(const RnArgs& A, const C_& C, int64_t sample) {
        uint64_t gate[4];
        vector8(A.gate, A.gate_each ? sample * A.c : 0, C, 1.f, gate);
        vector8(A.post_gamma, 0, C, 1.f, a);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = mul2(a[e], mul2(both(A.scale), gate[e]));
        vector8(A.pre_gamma, A.pre_each ? sample * A.c : 0, C, 1.f, g);
    }
};
// dx of B rows from the values d of dr, rh of r and u of dh; rows that are not there are zeros.
template <bool WIDE, int B, typename C_>
__device__ __forceinline__ void bwd_stream(const RnArgs& A, const C_& C, RowSum<WIDE>& sum, BwdVectors& V, const float4 (&st)[B], uint64_t (&d)[B][4],
                                           uint64_t (&rh)[B][4], uint64_t (&u)[B][4]) {
    float m[2 * B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
        uint64_t m0 = 0, m1 = 0;
        const uint64_t less = both(-st[k].z), wide = both(st[k].w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            rh[k][e] = mul2(add2(rh[k][e], less), wide);
            V.sc[e] = fma2(u[k][e], rh[k][e], V.sc[e]), V.sd[e] = add2(V.sd[e], u[k][e]);
            u[k][e] = mul2(u[k][e], V.g[e]);
            m0 = add2(m0, u[k][e]);
            m1 = fma2(u[k][e], rh[k][e], m1);
        }
        m[2 * k] = total(m0), m[2 * k + 1] = total(m1);
    }
    sum(m);
#pragma unroll
    for (int k = 0; k < B; ++k) {
        const uint64_t m0 = both(A.pre == CF_NORM_LAYER ? -m[2 * k] * A.inv_c : 0.f), m1 = both(-m[2 * k + 1] * A.inv_c), wide = both(st[k].w);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[k][e] = fma2(wide, fma2(rh[k][e], m1, add2(u[k][e], m0)), d[k][e]);
    }
}
// df (in d) from dx (in d) and the values w of f.
template <bool WIDE, int B, typename C_>
__device__ __forceinline__ void bwd_block(const RnArgs& A, const C_& C, RowSum<WIDE>& sum, BwdVectors& V, const float4 (&st)[B], uint64_t (&d)[B][4],
                                          uint64_t (&w)[B][4]) {
    float n[2 * B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
        uint64_t n0 = 0, n1 = 0;
        const uint64_t less = both(-st[k].x), wide = both(st[k].y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[k][e] = mul2(add2(w[k][e], less), wide);
            V.sa[e] = fma2(d[k][e], w[k][e], V.sa[e]), V.sb[e] = add2(V.sb[e], d[k][e]);
            d[k][e] = mul2(d[k][e], V.a[e]);
            n0 = add2(n0, d[k][e]);
            n1 = fma2(d[k][e], w[k][e], n1);
        }
        n[2 * k] = total(n0), n[2 * k + 1] = total(n1);
    }
    if (A.post == CF_NORM_NONE) return;
    sum(n);
#pragma unroll
    for (int k = 0; k < B; ++k) {
        const uint64_t n0 = both(A.post == CF_NORM_LAYER ? -n[2 * k] * A.inv_c : 0.f), n1 = both(-n[2 * k + 1] * A.inv_c), wide = both(st[k].y);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[k][e] = mul2(wide, fma2(w[k][e], n1, add2(d[k][e], n0)));
    }
}

// The block's sums to its part, in the order of its warps; `all` has room for 256 floats of each of `warps` warps.
template <bool WIDE, typename C_>
__device__ __forceinline__ void put_sums(const RnArgs& A, const C_& C, int T, BwdVectors& V, float* part, float* all, int warps) {
    float* to = part + (int64_t)blockIdx.x * 4 * A.c;
    auto put = [&](uint64_t (&q)[4], int which) {
        float v[8];
        spread(q, v);
        float* p = to + (int64_t)which * A.c;
        if (WIDE) {
            if (C.vec) {
                if (C.has(0)) {
                    float4* at = reinterpret_cast<float4*>(p + 8 * C.t);
                    at[0] = make_float4(v[0], v[1], v[2], v[3]), at[1] = make_float4(v[4], v[5], v[6], v[7]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (C.has(e)) p[C.at(e)] = v[e];
            }
            return;
        }
        const int warp = threadIdx.x >> 5;
        for (int o = T; o < 32; o <<= 1)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += __shfl_xor_sync(~0u, v[e], o);
        __syncthreads();
        if (warp < warps && (int)(threadIdx.x & 31) < T)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (C.has(e)) all[warp * 256 + C.at(e)] = v[e];
        __syncthreads();
        if ((int)threadIdx.x < A.c) {
            float s = 0.f;
            for (int w = 0; w < warps; ++w) s += all[w * 256 + threadIdx.x];
            p[threadIdx.x] = s;
        }
    };
    put(V.sa, 0), put(V.sb, 1), put(V.sc, 2), put(V.sd, 3);
}

template <typename S, typename F, bool WIDE, bool VEC>
__global__ void __launch_bounds__(WIDE ? kMostWide / 8 : kThreads, WIDE ? 1 : 2) rn_bwd_kernel(const RnArgs A, int T, const F* f, const S* r,
                                                                                              const float4* stats, const F* dh, const S* dr, S* dx,
                                                                                              F* df, float* part) {
    __shared__ float red[2][16][2 * kMostRows];
    __shared__ float all[WIDE ? 1 : kThreads / 32 * 256];
    Cols<VEC> C;
    const Place P = place_of<WIDE>(A, T, C);
    RowSum<WIDE> sum{red, 0, T};
    BwdVectors V(A, C, P.sample);
    const int64_t rounds = (P.to - (P.from - (WIDE ? 0 : (int)threadIdx.x / T)) + P.step - 1) / P.step;
    Raw<F> fn{}, dhn{};
    Raw<S> rn{}, drn{};
    float4 stn = make_float4(0.f, 1.f, 0.f, 1.f);
    auto fetch = [&](int64_t i) {
        const int64_t o = i * A.c;
        stn = make_float4(0.f, 1.f, 0.f, 1.f);
        fn = dhn = Raw<F>{}, rn = drn = Raw<S>{};  // zeros for what is not there
        if (i >= P.to) return;
        stn = __ldcg(stats + i);
        if (dh) rn = load8(r, o, C), dhn = load8(dh, o, C);
        if (dr) drn = load8(dr, o, C);
        if (f) fn = load8(f, o, C);
    };
    fetch(P.from);
    for (int64_t k = 0; k < rounds; ++k) {
        const int64_t i = P.from + k * P.step, o = i * A.c;
        const bool mine = i < P.to;
        uint64_t d[1][4], w[1][4];
        const float4 st[1] = {stn};
        unpack(drn, d[0]);
        unpack(fn, w[0]);
        if (A.pre != CF_NORM_NONE) {
            uint64_t rh[1][4], u[1][4];
            unpack(rn, rh[0]);
            unpack(dhn, u[0]);
            fetch(i + P.step);
            bwd_stream(A, C, sum, V, st, d, rh, u);
        } else {
            fetch(i + P.step);
        }
        if (dx && mine) store8(dx, o, C, d[0]);
        if (f) {
            bwd_block(A, C, sum, V, st, d, w);
            if (df && mine) store8(df, o, C, d[0]);
        }
    }
    if (part) put_sums<WIDE>(A, C, T, V, part, all, kThreads / 32);
}

// ------------------------------------------------------------------------------------------------ the same, fed by bulk copies
// A block's rows are one stretch of memory of each tensor, copied into stages of `high` rows: what is on its way does not depend on what
// registers hold.  Threads work on two rows at a time (ROWS), whose sums go together: a row's time is mostly the latency of those; but for
// the backward of rows that all threads share, which has the registers for one.  Rows of warps have a warp that copies; where all threads
// have a row, the first does, for the stage before, once all are through with it.  A row's sums of one barrier instead of two (of dv with
// the next row's of u) were slower: 302 us in place of 213 at 131072 x 512.
// Bulk copies begin and end at multiples of 16 bytes: where rows do not, a stage's first row lies up to 15 bytes into its room, and what
// is left of a tensor behind its last whole 16 bytes is copied value by value.
constexpr int kRingWarps = 15;
constexpr int kMostRing = 8;

struct RnRing {
    int high, stages;  // rows of a stage
    uint32_t stage_bytes;
    int* status;
    uint64_t wait_ns;
};
struct RnShared {
    uint64_t full[kMostRing], empty[kMostRing];
    int abort;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// What a stage holds, one after another: a row's bytes of each (0: not there), a multiple of 16 or `size` times so many values.
struct RnTensors {
    const char* at[5];
    int bytes[5], size[5];
    int64_t rows;
};
// A tensor's room in a stage.
__host__ __device__ inline int room_of(int high, int bytes) { return bytes ? (high * bytes + 30) & ~15 : 0; }
// The copies of one stage after another, by a warp: a lane to each tensor.
struct RingFill {
    int64_t i, end = 0;  // the next row; the tensor's bytes
    const char* at = nullptr;
    int mine = 0, size = 0, before = 0;
    int stage = 0;
    uint32_t parity = 1, issued = 0;
    __device__ __forceinline__ RingFill(const RnTensors& X, int high, int64_t from) : i(from) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            if (k < lane) before += room_of(high, X.bytes[k]);
            if (k == lane) at = X.at[k], mine = X.bytes[k], size = X.size[k];
        }
        end = X.rows * mine;
    }
    __device__ __forceinline__ bool next(const RnRing& R, RnShared& sh, uint8_t* ring, int64_t to) {
        const bool ok = mbar_wait(&sh.empty[stage], parity, &sh.abort, R.wait_ns, R.status, WAIT_PRODUCER_EMPTY);
        if (!__all_sync(~0u, ok)) return false;
        const int64_t first = i * mine, last = min(i + R.high, to) * mine, low = first & ~(int64_t)15;
        const int64_t high = min((last + 15) & ~(int64_t)15, end & ~(int64_t)15);
        uint8_t* dst = ring + stage * R.stage_bytes + before;
        for (int64_t b = high; b < last; b += size) {
            if (size == 4)
                *reinterpret_cast<float*>(dst + (b - low)) = *reinterpret_cast<const float*>(at + b);
            else
                *reinterpret_cast<uint16_t*>(dst + (b - low)) = *reinterpret_cast<const uint16_t*>(at + b);
        }
        const uint32_t bytes = __reduce_add_sync(~0u, (uint32_t)(high - low));
        __syncwarp();  // the arrival announces all lanes' values: a reduction orders no memory
        if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(&sh.full[stage], bytes);
        __syncwarp();
        if (high > low) bulk_load(dst, at + low, (uint32_t)(high - low), &sh.full[stage]);
        ++issued;
        i += R.high;
        if (++stage == R.stages) stage = 0, parity ^= 1;
        return true;
    }
    // after a wait that gave up: copies in flight end before the block leaves
    __device__ __forceinline__ void drain(const RnRing& R, RnShared& sh) const {
        if (*(volatile int*)&sh.abort && (threadIdx.x & 31) == 0)
            for (uint32_t k = issued > (uint32_t)R.stages ? issued - R.stages : 0; k < issued; ++k)
                mbar_wait_timed(&sh.full[k % R.stages], (k / R.stages) & 1, R.wait_ns);
    }
};

// Sets the block up; the rows of its chunk.
template <bool WIDE, typename C_>
__device__ __forceinline__ Place ring_begin(const RnArgs& A, int T, C_& C, const RnRing& R, RnShared& sh) {
    const int compute = WIDE ? T : 32 * kRingWarps;
    C.c = A.c, C.T = T, C.t = WIDE ? threadIdx.x : threadIdx.x & (T - 1);
    if (threadIdx.x == 0) {
        for (int k = 0; k < R.stages; ++k) mbar_init(&sh.full[k], 1), mbar_init(&sh.empty[k], compute / 32);
        sh.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    Place P;
    P.sample = blockIdx.x / A.chunks;
    P.from = P.sample * A.per + (blockIdx.x - P.sample * A.chunks) * A.chunk;
    P.to = min(min(P.from + A.chunk, (P.sample + 1) * A.per), A.rows);
    P.step = WIDE ? 1 : kRingWarps * 32 / T;
    return P;
}
// The thread's values of row k of a tensor's room, in a stage that begins with row i.
template <typename T_, typename C_>
__device__ __forceinline__ void from_stage(const uint8_t* room, bool there, const C_& C, int64_t i, int k, uint64_t (&v)[4]) {
    Raw<T_> raw{};
    if (C.vec) {
        if (there && C.has(0)) {
            const uint4* q = reinterpret_cast<const uint4*>(room + (k * C.c + 8 * C.t) * (int)sizeof(T_));
#pragma unroll
            for (int e = 0; e < (int)sizeof(T_) / 2; ++e) {
                const uint4 x = q[e];
                raw.u[4 * e] = x.x, raw.u[4 * e + 1] = x.y, raw.u[4 * e + 2] = x.z, raw.u[4 * e + 3] = x.w;
            }
        }
    } else if (there) {
        const T_* q = reinterpret_cast<const T_*>(room + ((int)(i * C.c * (int)sizeof(T_)) & 15)) + k * C.c;
        if (sizeof(T_) == 4) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (C.has(e)) raw.u[e % (2 * sizeof(T_))] = *reinterpret_cast<const uint32_t*>(q + C.at(e));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (C.has(e)) raw.u[e / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(q + C.at(e)) << 16 * (e & 1);
        }
    }
    unpack(raw, v);
}

// All threads' way through the stages: body(stage's bytes, first row of the stage that is the thread's, how many the stage has, the
// block's row that the stage begins with).  WIDE, where all threads meet in a row's sums, they leave together when one has given a
// wait up.
template <bool WIDE, int ROWS, typename B>
__device__ __forceinline__ void ring_run(const RnRing& R, const RnTensors& X, const Place& P, int T, RowSum<WIDE>& sum, RnShared& sh, uint8_t* ring,
                                         B body) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = WIDE ? 0 : warp * (32 / T), in = WIDE ? 0 : lane / T;
    RingFill fill(X, R.high, P.from);
    if (!WIDE && warp == kRingWarps) {
        while (fill.i < P.to && fill.next(R, sh, ring, P.to)) {}
        fill.drain(R, sh);
        return;
    }
    if (WIDE && warp == 0)
        for (int k = 0; k + 1 < R.stages && fill.i < P.to; ++k)
            if (!fill.next(R, sh, ring, P.to)) sum.failed = 1;
    int stage = 0;
    uint32_t parity = 0;
    for (int64_t i = P.from; i < P.to; i += R.high) {
        if (WIDE && warp == 0 && fill.i < P.to && !fill.next(R, sh, ring, P.to)) sum.failed = 1;
        const int rows = (int)min((int64_t)R.high, P.to - i);
        const bool ok = mbar_wait(&sh.full[stage], parity, &sh.abort, R.wait_ns, R.status, WAIT_MMA_FULL);
        if (!WIDE && !__all_sync(~0u, ok)) break;
        if (!ok) sum.failed = 1;
        for (int k = at; k < rows; k += ROWS * P.step) {
            body(ring + stage * R.stage_bytes, k + in, rows, i);
            if (WIDE && sum.failed) break;
        }
        if (WIDE && sum.failed) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);
        if (++stage == R.stages) stage = 0, parity ^= 1;
    }
    if (WIDE && warp == 0) fill.drain(R, sh);
}

template <typename S, typename F, bool WIDE, int ROWS, bool VEC>
__global__ void __launch_bounds__(512, 1) rn_fwd_ring_kernel(const RnArgs A, int T, const RnRing R, const S* x, const F* f, S* r, F* h, float4* stats) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RnShared sh;
    __shared__ float red[2][16][2 * kMostRows];
    Cols<VEC> C;
    const Place P = ring_begin<WIDE>(A, T, C, R, sh);
    const int row = A.c * (int)sizeof(S);
    const RnTensors X{{reinterpret_cast<const char*>(x), reinterpret_cast<const char*>(f)}, {row, f ? A.c * (int)sizeof(F) : 0},
                      {sizeof(S), sizeof(F)}, A.rows};
    const int of_f = room_of(R.high, row);
    RowSum<WIDE> sum{red, 0, T};
    const FwdVectors V(A, C, P.sample);
    ring_run<WIDE, ROWS>(R, X, P, T, sum, sh, ring, [&](const uint8_t* stage, int k, int rows, int64_t i) {
        uint64_t v[ROWS][4], w[ROWS][4];
        bool mine[ROWS];
#pragma unroll
        for (int b = 0; b < ROWS; ++b) {
            mine[b] = k + b * P.step < rows;
            from_stage<S>(stage, mine[b], C, i, k + b * P.step, v[b]);
            from_stage<F>(stage + of_f, f && mine[b], C, i, k + b * P.step, w[b]);
        }
        fwd_rows(A, C, sum, V, f != nullptr, i + k, P.step, mine, v, w, r, h, stats);
    });
}

template <typename S, typename F, bool WIDE, int ROWS, bool VEC>
__global__ void __launch_bounds__(512, 1) rn_bwd_ring_kernel(const RnArgs A, int T, const RnRing R, const F* f, const S* r, const float4* stats,
                                                           const F* dh, const S* dr, S* dx, F* df, float* part) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RnShared sh;
    __shared__ float red[2][16][2 * kMostRows];
    Cols<VEC> C;
    const Place P = ring_begin<WIDE>(A, T, C, R, sh);
    const int rs = A.c * (int)sizeof(S), rf = A.c * (int)sizeof(F);
    const RnTensors X{{reinterpret_cast<const char*>(r), reinterpret_cast<const char*>(dr), reinterpret_cast<const char*>(dh),
                       reinterpret_cast<const char*>(f), reinterpret_cast<const char*>(stats)},
                      {dh ? rs : 0, dr ? rs : 0, dh ? rf : 0, f ? rf : 0, 16}, {sizeof(S), sizeof(S), sizeof(F), sizeof(F), 4}, A.rows};
    const int o1 = room_of(R.high, X.bytes[0]), o2 = o1 + room_of(R.high, X.bytes[1]), o3 = o2 + room_of(R.high, X.bytes[2]);
    const int o4 = o3 + room_of(R.high, X.bytes[3]);
    BwdVectors V(A, C, P.sample);
    RowSum<WIDE> sum{red, 0, T};
    ring_run<WIDE, ROWS>(R, X, P, T, sum, sh, ring, [&](const uint8_t* stage, int k, int rows, int64_t i) {
        uint64_t d[ROWS][4];
        float4 st[ROWS];
        bool mine[ROWS];
#pragma unroll
        for (int b = 0; b < ROWS; ++b) {
            mine[b] = k + b * P.step < rows;
            st[b] = mine[b] ? *reinterpret_cast<const float4*>(stage + o4 + 16 * (k + b * P.step)) : make_float4(0.f, 1.f, 0.f, 1.f);
            from_stage<S>(stage + o1, dr && mine[b], C, i, k + b * P.step, d[b]);
        }
        if (A.pre != CF_NORM_NONE) {
            uint64_t rh[ROWS][4], u[ROWS][4];
#pragma unroll
            for (int b = 0; b < ROWS; ++b) {
                from_stage<S>(stage, mine[b], C, i, k + b * P.step, rh[b]);
                from_stage<F>(stage + o2, mine[b], C, i, k + b * P.step, u[b]);
            }
            bwd_stream(A, C, sum, V, st, d, rh, u);
        }
#pragma unroll
        for (int b = 0; b < ROWS; ++b)
            if (dx && mine[b]) store8(dx, (i + k + b * P.step) * A.c, C, d[b]);
        if (f) {
            uint64_t w[ROWS][4];
#pragma unroll
            for (int b = 0; b < ROWS; ++b) from_stage<F>(stage + o3, mine[b], C, i, k + b * P.step, w[b]);
            bwd_block(A, C, sum, V, st, d, w);
#pragma unroll
            for (int b = 0; b < ROWS; ++b)
                if (df && mine[b]) store8(df, (i + k + b * P.step) * A.c, C, d[b]);
        }
    });
    if (part == nullptr) return;
    __syncthreads();  // the stages are read, and hold the sums now
    put_sums<WIDE>(A, C, T, V, part, reinterpret_cast<float*>(ring), kRingWarps);
}

// ------------------------------------------------------------------------------------------------ longer rows
// Rows of any length, a block's threads with eight values each at a time, read again for each sum (from L1 or L2).
template <bool VEC>
__device__ __forceinline__ Cols<VEC> cols_at(int c, int first, int lanes, int lane) {
    Cols<VEC> C;
    C.c = c, C.T = lanes, C.t = VEC ? first / 8 + lane : first + lane;
    return C;
}
__device__ __forceinline__ void normed(uint64_t (&v)[4], float mean, float rstd) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = mul2(add2(v[e], both(-mean)), both(rstd));
}
template <bool VEC>
__device__ __forceinline__ void keep_own(const Cols<VEC>& C, uint64_t (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a, b;
        apart(v[e], a, b);
        v[e] = two(C.has(2 * e) ? a : 0.f, C.has(2 * e + 1) ? b : 0.f);
    }
}

template <typename S, typename F, bool VEC>
__global__ void __launch_bounds__(kThreads) rn_fwd_long_kernel(const RnArgs A, const S* x, const F* f, S* r, F* h, float4* stats) {
    __shared__ float2 red[kThreads / 32];
    constexpr int kStep = 8 * kThreads;
    for (int64_t i = blockIdx.x; i < A.rows; i += gridDim.x) {
        const int64_t o = i * A.c, sample = i / A.per;
        float2 sf = make_float2(0.f, 1.f), sr = sf;
        // r's values from column j0 on, f's normalised with sf
        auto value = [&](const Cols<VEC>& C, uint64_t (&v)[4]) {
            unpack(load8(x, o, C), v);
            if (!f) return;
            uint64_t w[4];
            unpack(load8(f, o, C), w);
            normed(w, sf.x, sf.y);
            const FwdVectors V(A, C, sample);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = add2(v[e], fma2(V.a[e], w[e], V.b[e]));
        };
        auto stats_of = [&](int kind, auto get, float2& st) {
            if (kind == CF_NORM_NONE) return;
            float mean = 0.f, s = 0.f;
            for (int pass = kind == CF_NORM_LAYER ? 0 : 1; pass < 2; ++pass) {
                s = 0.f;
                for (int j0 = 0; j0 < A.c; j0 += kStep) {
                    const Cols<VEC> C = cols_at<VEC>(A.c, j0, kThreads, threadIdx.x);
                    uint64_t v[4], q = 0;
                    get(C, v);
                    if (pass == 0) {
                        s += total(add2(add2(v[0], v[1]), add2(v[2], v[3])));
                        continue;
                    }
                    normed(v, mean, 1.f);
                    keep_own(C, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) q = fma2(v[e], v[e], q);
                    s += total(q);
                }
                s = block_sum(s, 0.f, red).x * A.inv_c;
                if (pass == 0) mean = s;
            }
            st = make_float2(mean, rsqrtf(s + A.eps));
        };
        if (f) stats_of(A.post, [&](const Cols<VEC>& C, uint64_t (&v)[4]) { unpack(load8(f, o, C), v); }, sf);
        stats_of(A.pre, value, sr);
        __syncthreads();  // all have read the row before r, which may be x, is written
        for (int j0 = 0; j0 < A.c; j0 += kStep) {
            const Cols<VEC> C = cols_at<VEC>(A.c, j0, kThreads, threadIdx.x);
            uint64_t v[4];
            value(C, v);
            if (r) store8(r, o, C, v);
            if (h) {
                const FwdVectors V(A, C, sample);
                normed(v, sr.x, sr.y);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = fma2(v[e], V.g[e], V.beta[e]);
                store8(h, o, C, v);
            }
        }
        if (stats && threadIdx.x == 0) stats[i] = make_float4(sf.x, sf.y, sr.x, sr.y);
    }
}

// dx of eight values of a row, from m = (mean u, mean u rh) (0, 0 and no norm: dr).
template <typename S, typename F, bool VEC>
__device__ __forceinline__ void dx8(const RnArgs& A, const Cols<VEC>& C, int64_t o, const S* r, const F* dh, const S* dr, const float4& st, float2 m,
                                    const uint64_t (&g)[4], uint64_t (&d)[4], uint64_t (&rh)[4], uint64_t (&u)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = rh[e] = u[e] = 0;
    if (dr) unpack(load8(dr, o, C), d);
    if (A.pre == CF_NORM_NONE) return;
    unpack(load8(r, o, C), rh);
    unpack(load8(dh, o, C), u);
    normed(rh, st.z, st.w);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = fma2(both(st.w), fma2(rh[e], both(-m.y), fma2(u[e], g[e], both(-m.x))), d[e]);
}

// The means that a row's gradients take.
template <typename S, typename F, bool VEC>
__global__ void __launch_bounds__(kThreads) rn_bwd_rows_kernel(const RnArgs A, const F* f, const S* r, const float4* stats, const F* dh, const S* dr,
                                                               float4* means) {
    __shared__ float2 red[kThreads / 32];
    constexpr int kStep = 8 * kThreads;
    for (int64_t i = blockIdx.x; i < A.rows; i += gridDim.x) {
        const int64_t o = i * A.c, sample = i / A.per;
        const float4 st = stats[i];
        float2 m = make_float2(0.f, 0.f), n = m;
        uint64_t d[4], rh[4], u[4];
        if (A.pre != CF_NORM_NONE) {
            for (int j0 = 0; j0 < A.c; j0 += kStep) {
                const Cols<VEC> C = cols_at<VEC>(A.c, j0, kThreads, threadIdx.x);
                const BwdVectors V(A, C, sample);
                dx8(A, C, o, r, dh, static_cast<const S*>(nullptr), st, m, V.g, d, rh, u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t t = mul2(u[e], V.g[e]);
                    m.x += total(t), m.y += total(mul2(t, rh[e]));
                }
            }
            m = block_sum(m.x, m.y, red);
            m.x = A.pre == CF_NORM_LAYER ? m.x * A.inv_c : 0.f;
            m.y *= A.inv_c;
        }
        if (A.post != CF_NORM_NONE) {
            for (int j0 = 0; j0 < A.c; j0 += kStep) {
                const Cols<VEC> C = cols_at<VEC>(A.c, j0, kThreads, threadIdx.x);
                const BwdVectors V(A, C, sample);
                uint64_t w[4];
                dx8(A, C, o, r, dh, dr, st, m, V.g, d, rh, u);
                unpack(load8(f, o, C), w);
                normed(w, st.x, st.y);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t t = mul2(d[e], V.a[e]);
                    n.x += total(t), n.y += total(mul2(t, w[e]));
                }
            }
            n = block_sum(n.x, n.y, red);
            n.x = A.post == CF_NORM_LAYER ? n.x * A.inv_c : 0.f;
            n.y *= A.inv_c;
        }
        if (threadIdx.x == 0) means[i] = make_float4(m.x, m.y, n.x, n.y);
    }
}

// dx, df and the chunk's sums over rows, from the rows' means: 256 columns to a block, a row to a warp.
template <typename S, typename F, bool VEC>
__global__ void __launch_bounds__(kThreads) rn_bwd_cols_kernel(const RnArgs A, const F* f, const S* r, const float4* stats, const F* dh, const S* dr,
                                                               const float4* means, S* dx, F* df, float* part) {
    __shared__ float all[kThreads / 32][256];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const Cols<VEC> C = cols_at<VEC>(A.c, blockIdx.y * 256, 32, lane);
    const int64_t sample = blockIdx.x / A.chunks;
    const int64_t from = sample * A.per + (blockIdx.x - sample * A.chunks) * A.chunk;
    const int64_t to = min(min(from + A.chunk, (sample + 1) * A.per), A.rows);
    BwdVectors V(A, C, sample);
    for (int64_t i = from + q; i < to; i += kThreads / 32) {
        const int64_t o = i * A.c;
        const float4 st = stats[i], m = means[i];
        uint64_t d[4], rh[4], u[4], w[4] = {};
        if (f) unpack(load8(f, o, C), w);
        dx8(A, C, o, r, dh, dr, st, make_float2(m.x, m.y), V.g, d, rh, u);
        normed(w, st.x, st.y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            V.sc[e] = fma2(u[e], rh[e], V.sc[e]), V.sd[e] = add2(V.sd[e], u[e]);
            V.sa[e] = fma2(d[e], w[e], V.sa[e]), V.sb[e] = add2(V.sb[e], d[e]);
        }
        if (dx) store8(dx, o, C, d);
        if (df) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[e] = mul2(d[e], V.a[e]);
                if (A.post != CF_NORM_NONE) d[e] = mul2(both(st.y), fma2(w[e], both(-m.w), add2(d[e], both(-m.z))));
            }
            store8(df, o, C, d);
        }
    }
    auto put = [&](const uint64_t (&p)[4], int which) {
        float v[8];
        spread(p, v);
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) all[q][VEC ? 8 * lane + e : lane + 32 * e] = v[e];
        __syncthreads();
        const int j = blockIdx.y * 256 + threadIdx.x;
        if (j >= A.c) return;
        float s = 0.f;
        for (int k = 0; k < kThreads / 32; ++k) s += all[k][threadIdx.x];
        part[(int64_t)blockIdx.x * 4 * A.c + (int64_t)which * A.c + j] = s;
    };
    put(V.sa, 0), put(V.sb, 1), put(V.sc, 2), put(V.sd, 3);
}

struct RnGrads {
    float *post_gamma, *post_beta, *gate, *pre_gamma, *pre_beta;
};

// The sums of 32 columns over rows [0, count) of v [][4][c], of the first two weighted by a row's weight: in warp 0.
constexpr int kSumWarps = 32;
template <typename W>
__device__ __forceinline__ float4 column_sums(const float* v, int64_t count, int c, int j, float4 (*red)[32], W weight) {
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < c) {
#pragma unroll 4
        for (int64_t i = q; i < count; i += kSumWarps) {
            const float* p = v + i * 4 * c + j;
            const float w = weight(i);
            s.x = fmaf(w, __ldcg(p), s.x);
            s.y = fmaf(w, __ldcg(p + c), s.y);
            s.z += __ldcg(p + 2 * (int64_t)c);
            s.w += __ldcg(p + 3 * (int64_t)c);
        }
    }
    red[q][lane] = s;
    __syncthreads();
    if (q == 0)
        for (int i = 1; i < kSumWarps; ++i) s.x += red[i][lane].x, s.y += red[i][lane].y, s.z += red[i][lane].z, s.w += red[i][lane].w;
    return s;
}
// These launches begin under the end of the one before.
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Each sample's sums from its chunks' (kept where vectors are shared between samples), and the gradients that are a sample's own.
__global__ void __launch_bounds__(32 * kSumWarps) rn_sample_kernel(const RnArgs A, const float* part, float* sums, const RnGrads G) {
    __shared__ float4 red[kSumWarps][32];
    wait_previous();
    const int j = blockIdx.y * 32 + (threadIdx.x & 31);
    const int64_t sample = blockIdx.x, c = A.c;
    const float4 s = column_sums(part + sample * A.chunks * 4 * c, A.chunks, A.c, j, red, [](int64_t) { return 1.f; });
    if (threadIdx.x >= 32 || j >= A.c) return;
    const bool one = A.samples == 1;
    if (!one) {
        float* p = sums + sample * 4 * c + j;
        p[0] = s.x, p[c] = s.y, p[2 * c] = s.z, p[3 * c] = s.w;
    }
    if (G.gate && (one || A.gate_each))
        G.gate[sample * c + j] = A.scale * (at_or(A.post_gamma, j, 1.f) * s.x + at_or(A.post_beta, j, 0.f) * s.y);
    if (one || A.pre_each) {
        if (G.pre_gamma) G.pre_gamma[sample * c + j] = s.z;
        if (G.pre_beta) G.pre_beta[sample * c + j] = s.w;
    }
    if (one) {
        const float g = A.scale * at_or(A.gate, j, 1.f);
        if (G.post_gamma) G.post_gamma[j] = g * s.x;
        if (G.post_beta) G.post_beta[j] = g * s.y;
    }
}

// The gradients of vectors that samples share.
__global__ void __launch_bounds__(32 * kSumWarps) rn_shared_kernel(const RnArgs A, const float* sums, const RnGrads G) {
    __shared__ float4 red[kSumWarps][32];
    wait_previous();
    const int j = blockIdx.x * 32 + (threadIdx.x & 31), c = A.c;
    const float4 s = column_sums(sums, A.samples, c, j, red, [&](int64_t i) { return A.gate_each ? at_or(A.gate, i * c + j, 1.f) : 1.f; });
    if (threadIdx.x >= 32 || j >= A.c) return;
    const float g = A.scale * (A.gate_each ? 1.f : at_or(A.gate, j, 1.f));
    if (G.post_gamma) G.post_gamma[j] = g * s.x;
    if (G.post_beta) G.post_beta[j] = g * s.y;
    if (G.gate && !A.gate_each) G.gate[j] = A.scale * (at_or(A.post_gamma, j, 1.f) * s.x + at_or(A.post_beta, j, 0.f) * s.y);
    if (!A.pre_each) {
        if (G.pre_gamma) G.pre_gamma[j] = s.z;
        if (G.pre_beta) G.pre_beta[j] = s.w;
    }
}

__global__ void __launch_bounds__(kThreads) rn_zero_kernel(float* p, int64_t count) {
    const int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    if (i < count) p[i] = 0.f;
}

// --------------------------------------------------------------------------------------------------------------------------- host
constexpr int kPlanSms = 152;  // work is cut for so many SMs: workspaces are laid out without asking the device

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
cf_status status_of() { return cudaGetLastError() == cudaSuccess ? CF_OK : CF_ERR_CUDA; }

// A launch that begins under the end of the one before it in the stream.
template <typename... P>
cf_status launch_after(const LaunchCtx& ctx, dim3 grid, void (*kernel)(P...), const std::common_type_t<P>&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kSumWarps);
    cfg.stream = ctx.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess ? CF_OK : (cudaGetLastError(), CF_ERR_CUDA);
}

RnArgs args_of(const cf_residual_norm_desc* d) {
    RnArgs A{};
    A.rows = d->rows, A.c = d->c, A.post = d->post, A.pre = d->pre;
    A.eps = d->eps, A.scale = d->scale, A.inv_c = 1.f / (float)d->c;
    A.per = d->rows_per_sample ? d->rows_per_sample : std::max<int64_t>(d->rows, 1);
    A.gate_each = (d->per_sample & CF_PER_SAMPLE_GATE) != 0, A.pre_each = (d->per_sample & CF_PER_SAMPLE_PRE) != 0;
    if (!d->per_sample) A.per = std::max<int64_t>(d->rows, 1);
    A.samples = (int)((d->rows + A.per - 1) / A.per);
    return A;
}
void vectors_of(RnArgs& A, const cf_residual_norm_vectors* v) {
    if (v == nullptr) return;
    A.post_gamma = v->post_gamma, A.post_beta = v->post_beta, A.gate = v->gate, A.pre_gamma = v->pre_gamma, A.pre_beta = v->pre_beta;
}
// Chunks of a sample's rows for about `blocks` blocks, of at least `least` rows.
void cut(RnArgs& A, int64_t blocks, int64_t least) {
    const int64_t per = std::min(A.per, A.rows);
    int64_t chunks = std::max<int64_t>(1, std::min((blocks + A.samples - 1) / std::max(A.samples, 1), per / least));
    A.chunk = (per + chunks - 1) / chunks;
    A.chunks = (int)((per + A.chunk - 1) / A.chunk);
}

// Threads of a row: up to 256 values a part of a warp, up to kMostWide a block, beyond that 0.
int threads_of(int c) {
    if (c > kMostWide) return 0;
    if (c > 256) return (c + 255) / 256 * 32;
    int T = 1;
    while (8 * T < c) T *= 2;
    return T;
}
// Blocks of the kernels without a ring that an SM holds, as many as their registers let it.
int per_sm(int T, int narrow) { return T <= 32 ? narrow : std::max(1, 512 / T); }
// And of those with one: a block of 15 warps and one that copies, or of T threads.
int ring_per_sm(int T) { return T <= 32 ? 1 : 512 / T; }

// Whether rows go through the ring: at least two rounds of rows to a block, and of a sample.  Fewer are quicker without (64 x 256,
// warm, forward 2.4 us without and 3.9 with it, backward 5.8 and 8.1); at the bound both take the same (9120 x 256 forward 5.8 and 6.0,
// backward 15.0 and 14.5); long ones, cold, are quicker with it (262144 x 256 forward 101 and 95, backward 183 and 153; 131072 x 512
// forward 117 and 107; 65536 x 515 203 and 132, 351 and 226).  The backward of rows that all threads of a block share, in whole words of
// eight, is not: its time is that of the block's sums (131072 x 512 195 us without and 213 with it, 16384 x 4096 218 and 220, of an fp32
// stream 246 and 243; warm 1216 x 4096 23 and 27).
bool ringed(const RnArgs& A, int T, bool backward) {
    if (backward && T > 32 && A.c % 8 == 0) return false;
    const int64_t step = T <= 32 ? kMostRows * (kRingWarps * 32 / T) : 2;
    return T && A.rows >= 2 * step * ring_per_sm(T) * kPlanSms && A.per >= 2 * step;
}
// A's rows cut for the kernel that takes them.
void cut_rows(RnArgs& A, int T, int narrow, bool backward) {
    if (ringed(A, T, backward))
        cut(A, (int64_t)kPlanSms * ring_per_sm(T), T <= 32 ? kRingWarps * 32 / T : 1);
    else
        cut(A, (int64_t)kPlanSms * per_sm(T, narrow), T <= 32 ? kThreads / T : 1);
}
RnRing ring_of(const LaunchCtx& ctx, const RnArgs& A, int T, int at_once, int per_row, int& shared) {
    RnRing R{};
    const int n = ring_per_sm(T), step = at_once * (T <= 32 ? kRingWarps * 32 / T : 1);
    const int room = 228 * 1024 / n - 1024 - 1024;  // what the system keeps of a block's, and the barriers
    R.high = std::max(1, (room / 5 - 288) / (per_row * step)) * step;  // five stages, or as many as fit of one round of rows
    if (3 * (R.high * per_row + 288) > room) R.high = step / at_once;
    R.high = (int)std::min<int64_t>(R.high, (A.chunk + step - 1) / step * step);
    R.stage_bytes = (uint32_t)((R.high * per_row + 5 * 32 + 127) / 128 * 128);
    R.stages = std::min(kMostRing, room / (int)R.stage_bytes);
    R.status = ctx.status, R.wait_ns = ctx.wait_ns;
    shared = std::max<int>(R.stages * R.stage_bytes, kRingWarps * 256 * 4);
    return R;
}

struct Layout {
    float4* means;
    float *part, *sums;
    size_t bytes;
};
Layout layout_of(const RnArgs& A, void* ws) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        void* p = static_cast<char*>(ws) + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    Layout L;
    L.means = static_cast<float4*>(take(A.c > kMostWide ? (size_t)A.rows * sizeof(float4) : 0));
    L.part = static_cast<float*>(take((size_t)A.samples * A.chunks * 4 * A.c * sizeof(float)));
    L.sums = static_cast<float*>(take(A.samples > 1 ? (size_t)A.samples * 4 * A.c * sizeof(float) : 0));
    L.bytes = std::max<size_t>(at, 256);
    return L;
}
RnArgs plan_bwd(const cf_residual_norm_desc* d) {
    RnArgs A = args_of(d);
    if (A.rows == 0) return A;
    const int T = threads_of(A.c);
    if (T)
        cut_rows(A, T, 2, true);
    else
        cut(A, std::max(1, kPlanSms * 4 * 256 / A.c), 8);
    return A;
}

cf_status check(const cf_residual_norm_desc* d) {
    if (d == nullptr || d->rows < 0 || d->c <= 0) return CF_ERR_INVALID_ARG;
    if (d->post < CF_NORM_NONE || d->post > CF_NORM_LAYER || d->pre < CF_NORM_NONE || d->pre > CF_NORM_LAYER) return CF_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->scale)) return CF_ERR_INVALID_ARG;
    if ((d->dtype != CF_DT_BF16 && d->dtype != CF_DT_F32) || (d->f_dtype != CF_DT_BF16 && d->f_dtype != CF_DT_F32)) return CF_ERR_INVALID_ARG;
    if ((d->per_sample & ~(CF_PER_SAMPLE_GATE | CF_PER_SAMPLE_PRE)) || d->rows_per_sample < 0) return CF_ERR_INVALID_ARG;
    if (d->dtype == CF_DT_BF16 && d->f_dtype == CF_DT_F32) return CF_ERR_UNSUPPORTED;
    if (d->c > 65536 || d->rows >= (int64_t)1 << 31) return CF_ERR_UNSUPPORTED;
    const int64_t per = d->rows_per_sample ? d->rows_per_sample : std::max<int64_t>(d->rows, 1);
    if (d->per_sample && (d->rows + per - 1) / per >= 1 << 24) return CF_ERR_UNSUPPORTED;
    return CF_OK;
}
bool vectors_ok(const cf_residual_norm_desc* d, const cf_residual_norm_vectors* v) {
    if (v == nullptr) return true;
    for (const float* p : {v->post_gamma, v->post_beta, v->gate, v->pre_gamma, v->pre_beta})
        if (!aligned16(p)) return false;
    if (d->post == CF_NORM_NONE && v->post_gamma) return false;
    if (d->pre == CF_NORM_NONE && v->pre_gamma) return false;
    return !(d->post != CF_NORM_LAYER && v->post_beta) && !(d->pre != CF_NORM_LAYER && v->pre_beta);
}

// f with the stream's and the blocks' types.
template <typename Fn>
cf_status with_types(const cf_residual_norm_desc* d, Fn f) {
    if (d->f_dtype == CF_DT_F32) return f(float{}, float{});
    if (d->dtype == CF_DT_F32) return f(float{}, uint16_t{});
    return f(uint16_t{}, uint16_t{});
}

}  // namespace
}  // namespace cf

using namespace cf;

extern "C" {

size_t cf_residual_norm_workspace_size(const cf_residual_norm_desc* desc) {
    if (check(desc) != CF_OK) return 0;
    return layout_of(plan_bwd(desc), nullptr).bytes;
}

cf_status cf_residual_norm_fwd(const cf_residual_norm_desc* desc, const void* x, const void* f, const cf_residual_norm_vectors* vectors,
                               void* r, void* h, float* stats, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    const bool pre = desc->pre != CF_NORM_NONE;
    if (!vectors_ok(desc, vectors) || (f == nullptr && (desc->post != CF_NORM_NONE || (vectors && vectors->gate)))) return CF_ERR_INVALID_ARG;
    if (desc->rows == 0) return CF_OK;
    if (!x || (h != nullptr) != pre || (!r && !h)) return CF_ERR_INVALID_ARG;
    for (const void* p : {x, f, (const void*)r, (const void*)h, (const void*)stats})
        if (!aligned16(p)) return CF_ERR_INVALID_ARG;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    RnArgs A = args_of(desc);
    vectors_of(A, vectors);
    return with_types(desc, [&](auto s, auto t) {
        using S = decltype(s);
        using F = decltype(t);
        const S* xs = static_cast<const S*>(x);
        const F* fs = static_cast<const F*>(f);
        float4* st4 = reinterpret_cast<float4*>(stats);
        if (const int T = threads_of(A.c); T) {
            cut_rows(A, T, 3, false);
            const unsigned blocks = (unsigned)(A.samples * A.chunks);
            if (ringed(A, T, false)) {
                int shared;
                const RnRing R = ring_of(ctx, A, T, 2, A.c * (int)(sizeof(S) + (f ? sizeof(F) : 0)), shared);
                auto kernel = A.c % 8 == 0 ? (T <= 32 ? rn_fwd_ring_kernel<S, F, false, 2, true> : rn_fwd_ring_kernel<S, F, true, 2, true>)
                                           : (T <= 32 ? rn_fwd_ring_kernel<S, F, false, 2, false> : rn_fwd_ring_kernel<S, F, true, 2, false>);
                if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared) != cudaSuccess) return status_of(), CF_ERR_CUDA;
                kernel<<<blocks, T <= 32 ? 32 * kRingWarps + 32 : T, shared, ctx.stream>>>(A, T, R, xs, fs, static_cast<S*>(r), static_cast<F*>(h), st4);
                return status_of();
            }
            auto kernel = A.c % 8 == 0 ? (T <= 32 ? rn_fwd_kernel<S, F, false, true> : rn_fwd_kernel<S, F, true, true>)
                                       : (T <= 32 ? rn_fwd_kernel<S, F, false, false> : rn_fwd_kernel<S, F, true, false>);
            kernel<<<blocks, T <= 32 ? kThreads : T, 0, ctx.stream>>>(A, T, xs, fs, static_cast<S*>(r), static_cast<F*>(h), st4);
            return status_of();
        }
        auto kernel = A.c % 8 == 0 ? rn_fwd_long_kernel<S, F, true> : rn_fwd_long_kernel<S, F, false>;
        kernel<<<(unsigned)std::min<int64_t>(A.rows, 8 * ctx.num_sms), kThreads, 0, ctx.stream>>>(A, xs, fs, static_cast<S*>(r), static_cast<F*>(h), st4);
        return status_of();
    });
}

cf_status cf_residual_norm_bwd(const cf_residual_norm_desc* desc, const void* f, const void* r, const cf_residual_norm_vectors* vectors,
                               const float* stats, const void* dh, const void* dr, void* dx, void* df,
                               const cf_residual_norm_vectors* grads, void* ws, size_t ws_bytes, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    const bool pre = desc->pre != CF_NORM_NONE;
    if (!vectors_ok(desc, vectors) || !vectors_ok(desc, grads)) return CF_ERR_INVALID_ARG;
    const bool sums = grads && (grads->post_gamma || grads->post_beta || grads->gate || grads->pre_gamma || grads->pre_beta);
    if (desc->rows) {
        if (!stats || (dh != nullptr) != pre || (pre && !r) || (!dh && !dr) || (!dx && !df && !sums)) return CF_ERR_INVALID_ARG;
        if (!f && (desc->post != CF_NORM_NONE || df || (vectors && vectors->gate) || (grads && grads->gate))) return CF_ERR_INVALID_ARG;
        for (const void* p : {f, r, (const void*)stats, dh, dr, (const void*)dx, (const void*)df, (const void*)ws})
            if (!aligned16(p)) return CF_ERR_INVALID_ARG;
    }
    RnArgs A = plan_bwd(desc);
    vectors_of(A, vectors);
    RnGrads G{};
    if (grads) G = RnGrads{grads->post_gamma, grads->post_beta, grads->gate, grads->pre_gamma, grads->pre_beta};
    const Layout L = layout_of(A, ws);
    if (desc->rows && (ws == nullptr || ws_bytes < L.bytes)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    if (desc->rows == 0) {
        // no samples either: a vector for each of them has no values
        const bool ge = A.gate_each, pe = A.pre_each;
        for (float* p : {G.post_gamma, G.post_beta, ge ? nullptr : G.gate, pe ? nullptr : G.pre_gamma, pe ? nullptr : G.pre_beta})
            if (p) {
                rn_zero_kernel<<<(A.c + kThreads - 1) / kThreads, kThreads, 0, ctx.stream>>>(p, A.c);
                if (const cf_status st = status_of(); st != CF_OK) return st;
            }
        return CF_OK;
    }
    return with_types(desc, [&](auto s, auto t) {
        using S = decltype(s);
        using F = decltype(t);
        const S *rs = static_cast<const S*>(r), *drs = static_cast<const S*>(dr);
        const F *fs = static_cast<const F*>(f), *dhs = static_cast<const F*>(dh);
        const float4* st4 = reinterpret_cast<const float4*>(stats);
        const unsigned tiles = (A.c + 31) / 32;  // of the sums' columns
        if (const int T = threads_of(A.c); T && ringed(A, T, true)) {
            int shared;
            const int per_row = A.c * (int)((dh ? sizeof(S) + sizeof(F) : 0) + (dr ? sizeof(S) : 0) + (f ? sizeof(F) : 0)) + 16;
            const RnRing R = ring_of(ctx, A, T, T <= 32 ? 2 : 1, per_row, shared);
            auto kernel = T > 32         ? rn_bwd_ring_kernel<S, F, true, 1, false>
                          : A.c % 8 == 0 ? rn_bwd_ring_kernel<S, F, false, 2, true>
                                         : rn_bwd_ring_kernel<S, F, false, 2, false>;
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared) != cudaSuccess) return status_of(), CF_ERR_CUDA;
            kernel<<<(unsigned)(A.samples * A.chunks), T <= 32 ? 32 * kRingWarps + 32 : T, shared, ctx.stream>>>(
                A, T, R, fs, rs, st4, dhs, drs, static_cast<S*>(dx), static_cast<F*>(df), sums ? L.part : nullptr);
        } else if (T) {
            auto kernel = A.c % 8 == 0 ? (T <= 32 ? rn_bwd_kernel<S, F, false, true> : rn_bwd_kernel<S, F, true, true>)
                                       : (T <= 32 ? rn_bwd_kernel<S, F, false, false> : rn_bwd_kernel<S, F, true, false>);
            kernel<<<(unsigned)(A.samples * A.chunks), T <= 32 ? kThreads : T, 0, ctx.stream>>>(A, T, fs, rs, st4, dhs, drs, static_cast<S*>(dx),
                                                                                               static_cast<F*>(df), sums ? L.part : nullptr);
        } else {
            const bool vec = A.c % 8 == 0;
            auto rows = vec ? rn_bwd_rows_kernel<S, F, true> : rn_bwd_rows_kernel<S, F, false>;
            auto cols = vec ? rn_bwd_cols_kernel<S, F, true> : rn_bwd_cols_kernel<S, F, false>;
            rows<<<(unsigned)std::min<int64_t>(A.rows, 8 * ctx.num_sms), kThreads, 0, ctx.stream>>>(A, fs, rs, st4, dhs, drs, L.means);
            if (const cf_status st = status_of(); st != CF_OK) return st;
            cols<<<dim3((unsigned)(A.samples * A.chunks), (A.c + 255) / 256), kThreads, 0, ctx.stream>>>(
                A, fs, rs, st4, dhs, drs, L.means, static_cast<S*>(dx), static_cast<F*>(df), L.part);
        }
        if (const cf_status st = status_of(); st != CF_OK || !sums) return st;
        if (const cf_status st = launch_after(ctx, dim3((unsigned)A.samples, tiles), rn_sample_kernel, A, L.part, L.sums, G); st != CF_OK || A.samples == 1)
            return st;
        return launch_after(ctx, dim3(tiles), rn_shared_kernel, A, L.sums, G);
    });
}

}  // extern "C"
