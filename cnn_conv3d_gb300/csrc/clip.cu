// clip.cu -- the global norm of a list of gradients, clipping by it, and the Adam step of a list with clipped gradients, with
// their entry points.
//
// The norm has to be known before the first gradient is scaled, so a call is two launches for any number of tensors: one that sums
// the squares, a part of all values to a block, and one that joins the parts, in every block alike, and applies the factor.  Both
// are bound by memory (Adam: 30 bytes a parameter besides the norm's 4), so what counts is that every block has the same number
// of bytes and keeps loads in flight.  The second launch begins under the end of the first and walks each block's values backwards,
// since the last ones read are those that L2 still has.  43M parameters: 244 us of Adam with the norm (6.0 TB/s, the gradients' second
// reading counted); 2.9M values' norm 7.6 us in a graph, of which the bytes are 1.7.
//
// Squares are summed in fp32 sixteen at a time and in 64 bits from there; a sum of sixteen that overflowed or came close to fp32's
// smallest values is taken again in 64 bits, which hold the square of any fp32 value.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "cf_internal.h"
#include "cf_ptx.cuh"

namespace cf {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 16;                    // values of a thread at a time
constexpr int kItem = kThreads * kUnit;      // values of a block at a time
constexpr int kNormBlocks = 6, kApplyBlocks = 4;  // resident on an SM
constexpr float kClipEps = 1e-6f;

// A tensor of the list.  Items are counted over the whole launch; `head` values come before the first that starts at 16 bytes.
struct Grad {
    const void* g;
    int64_t count;
    int32_t first;
    int16_t f32, head;
};
struct Param {
    float *w, *m, *v;
    uint16_t* w16;
    const float* g;
    int64_t count;
    int32_t first;
    int16_t vec, head;  // vec: all five tensors have their first aligned value at `head`
};
// As many as the arguments of a launch hold (32764 bytes), and few for short lists, whose launch is cheaper.
template <typename E, int CAP>
struct List {
    E e[CAP];
    int count, items;
};

__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The entry that item `at` belongs to.
template <typename E, int CAP>
__device__ __forceinline__ int entry_of(const List<E, CAP>& L, int at) {
    int lo = 0, hi = L.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (L.e[mid].first <= at)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ void range_of(int items, int& from, int& to) {
    from = (int)((int64_t)items * blockIdx.x / gridDim.x);
    to = (int)((int64_t)items * (blockIdx.x + 1) / gridDim.x);
}

__device__ __forceinline__ float value_of(const void* g, int f32, int64_t i) {
    return f32 ? static_cast<const float*>(g)[i] : bf16_bits_to_float(static_cast<const uint16_t*>(g)[i]);
}
__device__ __forceinline__ double squares(const float (&x)[kUnit]) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kUnit; ++i) s[i & 3] = fmaf(x[i], x[i], s[i & 3]);
    const float t = (s[0] + s[1]) + (s[2] + s[3]);
    if (t >= 0x1p-100f && t <= 0x1p126f) return (double)t;
    float any = 0.f;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) any = fmaxf(any, fabsf(x[i]));
    if (any == 0.f && t == 0.f) return 0.0;
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) d += (double)x[i] * (double)x[i];
    return d;
}

// 16 values from `from` on, vectors of 16 bytes a block's width apart: register 4 e + q (fp32), 8 e + q (bf16).
__device__ __forceinline__ void load_unit(const Grad& G, int64_t from, float (&x)[kUnit]) {
    if (G.f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(G.g) + from) + threadIdx.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 v = p[e * kThreads];
            x[4 * e] = v.x, x[4 * e + 1] = v.y, x[4 * e + 2] = v.z, x[4 * e + 3] = v.w;
        }
    } else {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(G.g) + from) + threadIdx.x;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint4 v = p[e * kThreads];
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                x[8 * e + 2 * q] = __uint_as_float(u[q] << 16);
                x[8 * e + 2 * q + 1] = __uint_as_float(u[q] & 0xFFFF0000u);
            }
        }
    }
}

// Sum over the block, in thread 0.
__device__ __forceinline__ double block_sum(double s, double* red) {
    for (int o = 16; o; o >>= 1) s += __shfl_down_sync(~0u, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int i = 1; i < kThreads / 32; ++i) s += red[i];
    return s;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kNormBlocks) clip_norm_kernel(const __grid_constant__ List<Grad, CAP> L, double* part) {
    __shared__ double red[kThreads / 32];
    start_next();
    int from, to;
    range_of(L.items, from, to);
    double s = 0.0;
    int i = entry_of(L, from);
    for (int at = from; at < to; ++at) {
        while (i + 1 < L.count && L.e[i + 1].first <= at) ++i;
        const Grad& G = L.e[i];
        const int64_t body = G.head + (int64_t)(at - G.first) * kItem;
        float x[kUnit];
        if (body + kItem <= G.count) {
            load_unit(G, body, x);
            s += squares(x);
        } else {
#pragma unroll
            for (int e = 0; e < kUnit; ++e) {
                const int64_t j = body + e * kThreads + threadIdx.x;
                x[e] = j < G.count ? value_of(G.g, G.f32, j) : 0.f;
            }
            s += squares(x);
        }
        if (at == G.first && (int)threadIdx.x < G.head) {
            const double d = threadIdx.x < G.count ? (double)value_of(G.g, G.f32, threadIdx.x) : 0.0;
            s += d * d;
        }
    }
    s = block_sum(s, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm and the factor from the parts, the same in every block.
__device__ __forceinline__ float2 join(const double* part, int parts, float max_norm, double* red) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += __ldcg(part + i);
    s = block_sum(s, red);
    if (threadIdx.x == 0) red[0] = s;
    __syncthreads();
    const float norm = (float)sqrt(red[0]);
    const float f = isinf(norm) ? 0.f : max_norm / (norm + kClipEps);  // also where max_norm is infinite
    return make_float2(norm, f < 1.f || f != f ? f : 1.f);
}

__global__ void __launch_bounds__(kThreads) clip_factor_kernel(const double* part, int parts, float max_norm, float* out) {
    __shared__ double red[kThreads / 32];
    wait_previous();
    const float2 r = join(part, parts, max_norm, red);
    if (threadIdx.x == 0) out[0] = r.x, out[1] = r.y;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kApplyBlocks) clip_scale_kernel(const __grid_constant__ List<Grad, CAP> L, const double* part, int parts,
                                                              float max_norm, float* out) {
    __shared__ double red[kThreads / 32];
    wait_previous();
    const float2 r = join(part, parts, max_norm, red);
    if (out && blockIdx.x == 0 && threadIdx.x == 0) out[0] = r.x, out[1] = r.y;
    if (r.y == 1.f) return;
    int from, to;
    range_of(L.items, from, to);
    if (from == to) return;
    int i = entry_of(L, to - 1);
    for (int at = to - 1; at >= from; --at) {
        while (L.e[i].first > at) --i;
        const Grad& G = L.e[i];
        const int64_t body = G.head + (int64_t)(at - G.first) * kItem;
        if (body + kItem <= G.count) {
            float x[kUnit];
            load_unit(G, body, x);
#pragma unroll
            for (int e = 0; e < kUnit; ++e) x[e] *= r.y;
            if (G.f32) {
                float4* p = reinterpret_cast<float4*>((float*)G.g + body) + threadIdx.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e * kThreads] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            } else {
                uint4* p = reinterpret_cast<uint4*>((uint16_t*)G.g + body) + threadIdx.x;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    p[e * kThreads] = make_uint4(pack_bf16x2(x[8 * e], x[8 * e + 1]), pack_bf16x2(x[8 * e + 2], x[8 * e + 3]),
                                                 pack_bf16x2(x[8 * e + 4], x[8 * e + 5]), pack_bf16x2(x[8 * e + 6], x[8 * e + 7]));
            }
        }
        const int64_t rest = body + kItem <= G.count ? G.count : body;
        auto one = [&](int64_t j) {
            const float x = value_of(G.g, G.f32, j) * r.y;
            if (G.f32)
                ((float*)G.g)[j] = x;
            else
                ((uint16_t*)G.g)[j] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        };
        for (int64_t j = rest + threadIdx.x; j < G.count; j += kThreads) one(j);
        if (at == G.first && threadIdx.x < min((int64_t)G.head, G.count)) one(threadIdx.x);
    }
}

struct AdamScalars {
    float beta1, beta2, rest1, rest2;  // rest: 1 - beta, which in fp32 would be off by 1e-5 of itself for 0.999
    float decay, step, eps, c2;        // decay = lr weight_decay, step = lr / (1 - beta1^t), c2 = 1 / (1 - beta2^t)
    float max_norm;
};
__device__ __forceinline__ void adam_one(const AdamScalars& S, float factor, float g, float& w, float& m, float& v) {
    g *= factor;
    m = fmaf(S.beta1, m, S.rest1 * g);
    v = fmaf(S.beta2, v, S.rest2 * g * g);
    w = fmaf(-S.step, m / (sqrtf(v * S.c2) + S.eps), fmaf(-S.decay, w, w));
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kApplyBlocks) clip_adam_kernel(const __grid_constant__ List<Param, CAP> L, const AdamScalars S,
                                                             const double* part, int parts, float* out) {
    __shared__ double red[kThreads / 32];
    wait_previous();
    float factor = 1.f;
    if (parts) {
        const float2 r = join(part, parts, S.max_norm, red);
        if (out && blockIdx.x == 0 && threadIdx.x == 0) out[0] = r.x, out[1] = r.y;
        factor = r.y;
    }
    int from, to;
    range_of(L.items, from, to);
    if (from == to) return;
    int i = entry_of(L, to - 1);
    for (int at = to - 1; at >= from; --at) {
        while (L.e[i].first > at) --i;
        const Param& P = L.e[i];
        int64_t body = P.head + (int64_t)(at - P.first) * kItem;
        const int64_t end = min(body + kItem, P.count);
        if (P.vec && body + kItem <= P.count) {
#pragma unroll 2
            for (int e = 0; e < kUnit / 4; ++e) {
                const int64_t j = body + 4 * (e * kThreads + threadIdx.x);
                const float4 g = *reinterpret_cast<const float4*>(P.g + j);
                float4 w = *reinterpret_cast<const float4*>(P.w + j);
                float4 m = *reinterpret_cast<const float4*>(P.m + j);
                float4 v = *reinterpret_cast<const float4*>(P.v + j);
                adam_one(S, factor, g.x, w.x, m.x, v.x);
                adam_one(S, factor, g.y, w.y, m.y, v.y);
                adam_one(S, factor, g.z, w.z, m.z, v.z);
                adam_one(S, factor, g.w, w.w, m.w, v.w);
                *reinterpret_cast<float4*>(P.w + j) = w;
                *reinterpret_cast<float4*>(P.m + j) = m;
                *reinterpret_cast<float4*>(P.v + j) = v;
                if (P.w16) *reinterpret_cast<uint2*>(P.w16 + j) = make_uint2(pack_bf16x2(w.x, w.y), pack_bf16x2(w.z, w.w));
            }
            body = end;
        }
        auto one = [&](int64_t j) {
            float w = P.w[j], m = P.m[j], v = P.v[j];
            adam_one(S, factor, P.g[j], w, m, v);
            P.w[j] = w, P.m[j] = m, P.v[j] = v;
            if (P.w16) P.w16[j] = __bfloat16_as_ushort(__float2bfloat16_rn(w));
        };
        for (int64_t j = body + threadIdx.x; j < end; j += kThreads) one(j);
        if (at == P.first && threadIdx.x < min((int64_t)P.head, P.count)) one(threadIdx.x);
    }
}

// --------------------------------------------------------------------------------------------------------------------------- host
cf_status cuda_error() {
    cudaGetLastError();
    return CF_ERR_CUDA;
}

// Values before the first that starts at 16 bytes.
int head_of(const void* p, int size) { return (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16) / size; }
int64_t items_of(int64_t count, int head) { return std::max<int64_t>(1, (count - head + kItem - 1) / kItem); }

bool grad_ok(const cf_grad& g) {
    if (g.count < 0 || (g.dtype != CF_DT_BF16 && g.dtype != CF_DT_F32)) return false;
    if (g.count == 0) return true;
    return g.g != nullptr && reinterpret_cast<uintptr_t>(g.g) % (g.dtype == CF_DT_F32 ? 4 : 2) == 0;
}
bool param_ok(const cf_adam_param& p) {
    if (p.count < 0) return false;
    if (p.count == 0) return true;
    if (!p.w || !p.g || !p.m || !p.v) return false;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.w) | reinterpret_cast<uintptr_t>(p.g) | reinterpret_cast<uintptr_t>(p.m) |
                           reinterpret_cast<uintptr_t>(p.v);
    return bits % 4 == 0 && reinterpret_cast<uintptr_t>(p.w_bf16) % 2 == 0;
}
template <typename P, typename F>
cf_status check(int32_t count, const P* p, F ok) {
    if (count < 0 || (count > 0 && p == nullptr)) return CF_ERR_INVALID_ARG;
    double items = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (!ok(p[i])) return CF_ERR_INVALID_ARG;
        items += (double)p[i].count / kItem + 1;
    }
    return items < 1e9 ? CF_OK : CF_ERR_UNSUPPORTED;
}

Grad entry(const cf_grad& g) {
    const int f32 = g.dtype == CF_DT_F32;
    return Grad{g.g, g.count, 0, (int16_t)f32, (int16_t)head_of(g.g, f32 ? 4 : 2)};
}
Grad entry_g(const cf_adam_param& p) { return Grad{p.g, p.count, 0, 1, (int16_t)head_of(p.g, 4)}; }
Param entry(const cf_adam_param& p) {
    const int head = head_of(p.w, 4);
    const bool vec = head_of(p.g, 4) == head && head_of(p.m, 4) == head && head_of(p.v, 4) == head &&
                     (reinterpret_cast<uintptr_t>(p.w_bf16) + 2 * (p.w_bf16 ? head : 0)) % 8 == 0;
    return Param{p.w, p.m, p.v, p.w_bf16, p.g, p.count, 0, (int16_t)vec, (int16_t)(vec ? head : 0)};
}

constexpr int kFew = 32, kManyGrads = 1024, kManyParams = 480;
static_assert(sizeof(List<Grad, kManyGrads>) + 64 <= 32764 && sizeof(List<Param, kManyParams>) + 128 <= 32764, "arguments of a launch");

int blocks_of(int items, int per_sm, int sms) { return std::min(items, per_sm * sms); }

// A launch that begins under the end of the one before it in the stream.
template <typename K, typename... A>
cf_status launch(cudaStream_t stream, int blocks, bool after, K kernel, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? CF_OK : cuda_error();
}

// The list in launches of `cap` entries: f(entries, how many, items).
template <typename E, typename F>
cf_status in_parts(std::vector<E>& all, int few, int many, F f) {
    const int cap = (int)all.size() <= few ? few : many;
    for (size_t i = 0; i < all.size(); i += cap) {
        const int n = (int)std::min<size_t>(cap, all.size() - i);
        int64_t items = 0;
        for (int j = 0; j < n; ++j) {
            all[i + j].first = (int32_t)items;
            items += items_of(all[i + j].count, all[i + j].head);
        }
        if (const cf_status st = f(&all[i], n, (int)items, cap == few); st != CF_OK) return st;
    }
    return CF_OK;
}
template <int CAP, typename E>
void fill(List<E, CAP>& L, const E* e, int n, int items) {
    std::copy(e, e + n, L.e);
    L.count = n, L.items = items;
}

// Parts of the sum that a list of so many entries leaves at most.
size_t parts_bytes(int32_t count, int sms) {
    const size_t launches = count <= kFew ? 1 : ((size_t)count + kManyGrads - 1) / kManyGrads;
    return std::max<size_t>(launches, 1) * kNormBlocks * sms * sizeof(double);
}
constexpr int kPlanSms = 160;  // workspaces are sized without asking the device

cf_status norm_parts(const LaunchCtx& ctx, std::vector<Grad>& grads, double* part, int& parts) {
    parts = 0;
    return in_parts(grads, kFew, kManyGrads, [&](Grad* e, int n, int items, bool few) {
        const int blocks = blocks_of(items, kNormBlocks, std::min(ctx.num_sms, kPlanSms));
        double* to = part + parts;
        parts += blocks;
        if (few) {
            List<Grad, kFew> L;
            fill(L, e, n, items);
            return launch(ctx.stream, blocks, false, clip_norm_kernel<kFew>, L, to);
        }
        List<Grad, kManyGrads> L;
        fill(L, e, n, items);
        return launch(ctx.stream, blocks, false, clip_norm_kernel<kManyGrads>, L, to);
    });
}

cf_status grad_call(int32_t count, const cf_grad* grads, float max_norm, float* out, void* ws, size_t ws_bytes, void* stream, bool scale) {
    if (!(max_norm >= 0.f) || out == nullptr || reinterpret_cast<uintptr_t>(out) % 4 || reinterpret_cast<uintptr_t>(ws) % 16)
        return CF_ERR_INVALID_ARG;
    if (const cf_status st = check(count, grads, grad_ok); st != CF_OK) return st;
    if (ws == nullptr || ws_bytes < cf_grad_workspace_size(count, grads)) return CF_ERR_WORKSPACE;
    std::vector<Grad> all;
    for (int32_t i = 0; i < count; ++i)
        if (grads[i].count) all.push_back(entry(grads[i]));
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    double* part = static_cast<double*>(ws);
    int parts;
    if (const cf_status st = norm_parts(ctx, all, part, parts); st != CF_OK) return st;
    if (!scale || all.empty()) return launch(ctx.stream, 1, !all.empty(), clip_factor_kernel, part, parts, max_norm, out);
    bool first = true;
    return in_parts(all, kFew, kManyGrads, [&](Grad* e, int n, int items, bool few) {
        const int blocks = blocks_of(items, kApplyBlocks, ctx.num_sms);
        // only the first may begin early: those after it would run beside the norm's launches too, whose parts they read
        const bool after = first;
        float* to = first ? out : nullptr;
        first = false;
        if (few) {
            List<Grad, kFew> L;
            fill(L, e, n, items);
            return launch(ctx.stream, blocks, after, clip_scale_kernel<kFew>, L, part, parts, max_norm, to);
        }
        List<Grad, kManyGrads> L;
        fill(L, e, n, items);
        return launch(ctx.stream, blocks, after, clip_scale_kernel<kManyGrads>, L, part, parts, max_norm, to);
    });
}

}  // namespace
}  // namespace cf

using namespace cf;

extern "C" {

size_t cf_grad_workspace_size(int32_t count, const cf_grad* grads) {
    return check(count, grads, grad_ok) == CF_OK ? parts_bytes(count, kPlanSms) : 0;
}

cf_status cf_grad_norm(int32_t count, const cf_grad* grads, float max_norm, float* out, void* ws, size_t ws_bytes, void* stream) try {
    return grad_call(count, grads, max_norm, out, ws, ws_bytes, stream, false);
} catch (const std::bad_alloc&) {  // the list
    return CF_ERR_UNSUPPORTED;
}

cf_status cf_clip_grads(int32_t count, const cf_grad* grads, float max_norm, float* out, void* ws, size_t ws_bytes, void* stream) try {
    return grad_call(count, grads, max_norm, out, ws, ws_bytes, stream, true);
} catch (const std::bad_alloc&) {  // the list
    return CF_ERR_UNSUPPORTED;
}

size_t cf_clip_adam_workspace_size(int32_t count, const cf_adam_param* params) {
    return check(count, params, param_ok) == CF_OK ? parts_bytes(count, kPlanSms) : 0;
}

cf_status cf_clip_adam_step(int32_t count, const cf_adam_param* params, const cf_adam_hyper* h, float* out, void* ws, size_t ws_bytes,
                            void* stream) try {
    if (h == nullptr || !(h->beta1 >= 0 && h->beta1 < 1 && h->beta2 >= 0 && h->beta2 < 1 && h->eps >= 0 && h->max_norm >= 0) ||
        h->t < 1 || !std::isfinite(h->lr) || !std::isfinite(h->weight_decay) || !std::isfinite(h->eps))
        return CF_ERR_INVALID_ARG;
    const bool clip = h->max_norm > 0;
    if ((clip && out == nullptr) || reinterpret_cast<uintptr_t>(out) % 4 || reinterpret_cast<uintptr_t>(ws) % 16) return CF_ERR_INVALID_ARG;
    if (const cf_status st = check(count, params, param_ok); st != CF_OK) return st;
    if (clip && (ws == nullptr || ws_bytes < parts_bytes(count, kPlanSms))) return CF_ERR_WORKSPACE;
    std::vector<Grad> grads;
    std::vector<Param> all;
    for (int32_t i = 0; i < count; ++i)
        if (params[i].count) grads.push_back(entry_g(params[i])), all.push_back(entry(params[i]));
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    double* part = static_cast<double*>(ws);
    int parts = 0;
    if (clip) {
        if (const cf_status st = norm_parts(ctx, grads, part, parts); st != CF_OK) return st;
        if (all.empty()) return launch(ctx.stream, 1, false, clip_factor_kernel, part, 0, (float)h->max_norm, out);
    }
    AdamScalars S;
    S.beta1 = (float)h->beta1, S.beta2 = (float)h->beta2;
    S.rest1 = (float)(1 - h->beta1), S.rest2 = (float)(1 - h->beta2);
    S.decay = (float)(h->lr * h->weight_decay), S.step = (float)(h->lr / (1 - std::pow(h->beta1, (double)h->t)));
    S.eps = (float)h->eps, S.c2 = (float)(1 / (1 - std::pow(h->beta2, (double)h->t)));
    S.max_norm = (float)h->max_norm;
    bool first = clip;
    return in_parts(all, kFew, kManyParams, [&](Param* e, int n, int items, bool few) {
        const int blocks = blocks_of(items, kApplyBlocks, ctx.num_sms);
        const bool after = first;  // as in grad_call
        float* to = first ? out : nullptr;
        first = false;
        if (few) {
            List<Param, kFew> L;
            fill(L, e, n, items);
            return launch(ctx.stream, blocks, after, clip_adam_kernel<kFew>, L, S, part, parts, to);
        }
        List<Param, kManyParams> L;
        fill(L, e, n, items);
        return launch(ctx.stream, blocks, after, clip_adam_kernel<kManyParams>, L, S, part, parts, to);
    });
} catch (const std::bad_alloc&) {  // the list
    return CF_ERR_UNSUPPORTED;
}

}  // extern "C"
