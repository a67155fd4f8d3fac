// linear.cu -- matrix products of bf16 rows with bias, activation and residual in the epilogue (forward), with the activation's
// derivative in it (backward data), and summed over the rows (backward weight), with their entry points.
//
// The products run in linear_gemm.cuh's kernel; here are its plans, the copies of operands whose rows TMA cannot fetch (they start
// at no multiple of 16 bytes), the activation's own backward and the checks.
#include <algorithm>
#include <cmath>

#include "linear_gemm.cuh"

namespace cf {
namespace {

// [rows][width] at any pitch as rows of `to` values, a multiple of 8; what is behind a row's end is not read by anyone.
__global__ void __launch_bounds__(256) linear_pack_kernel(const uint16_t* src, int64_t rows, int width, int64_t pitch, uint16_t* dst, int to) {
    const int per = to / 8;
    for (int64_t e = blockIdx.x * (int64_t)256 + threadIdx.x; e < rows * per; e += (int64_t)gridDim.x * 256) {
        const int64_t i = e / per;
        const int j = (int)(e - i * per) * 8;
        uint32_t u[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) u[x] = j + x < width ? src[i * pitch + j + x] : 0;
        *reinterpret_cast<uint4*>(dst + i * to + j) = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
    }
}

// dz = scale dy act'(pre), eight values of a row at a time (VEC: which begin at 16 bytes).  Memory bounds it.
template <bool VEC>
__global__ void __launch_bounds__(256) linear_act_bwd_kernel(const void* dy, const uint16_t* pre, uint16_t* dz, int64_t rows, int n, int64_t pitch,
                                                             const __grid_constant__ LinEpi E) {
    const int per = (n + 7) / 8;
    for (int64_t e = blockIdx.x * (int64_t)256 + threadIdx.x; e < rows * per; e += (int64_t)gridDim.x * 256) {
        const int64_t i = e / per;
        const int j = (int)(e - i * per) * 8;
        const int64_t o = i * pitch + j;
        float d[8], z[8];
        if (VEC) {
            const uint4 q = *reinterpret_cast<const uint4*>(pre + o);
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) z[2 * x] = __uint_as_float(u[x] << 16), z[2 * x + 1] = __uint_as_float(u[x] & 0xFFFF0000u);
            if (E.f32) {
                const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(dy) + o);
                const float4 a = p[0], b = p[1];
                d[0] = a.x, d[1] = a.y, d[2] = a.z, d[3] = a.w, d[4] = b.x, d[5] = b.y, d[6] = b.z, d[7] = b.w;
            } else {
                const uint4 p = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(dy) + o);
                const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) d[2 * x] = __uint_as_float(w[x] << 16), d[2 * x + 1] = __uint_as_float(w[x] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const bool in = j + x < n;
                z[x] = in ? bf16_bits_to_float(pre[o + x]) : 0.f;
                d[x] = !in ? 0.f : E.f32 ? static_cast<const float*>(dy)[o + x] : bf16_bits_to_float(static_cast<const uint16_t*>(dy)[o + x]);
            }
        }
        times_grad(E, z, d);
#pragma unroll
        for (int x = 0; x < 8; ++x) d[x] *= E.scale;
        if (VEC) {
            *reinterpret_cast<uint4*>(dz + o) = make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]), pack_bf16x2(d[4], d[5]), pack_bf16x2(d[6], d[7]));
        } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (j + x < n) dz[o + x] = __bfloat16_as_ushort(__float2bfloat16_rn(d[x]));
        }
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

constexpr int kMostSummed = 24;  // blocks whose sum the tensor cores take for an fp32 result
constexpr int kPlanSms = 152;  // work is cut for so many SMs: workspaces are laid out without asking the device

// An operand as it lies in memory: `rows` rows of `width` values, the contracted axis along them (K-major) or across.
struct Side {
    int64_t rows, width, pitch;
    bool mn;
    bool packed() const { return pitch % 8 != 0; }
    int64_t kept() const { return packed() ? (width + 7) / 8 * 8 : pitch; }
    size_t bytes() const { return packed() ? ((size_t)rows * kept() * 2 + 255) / 256 * 256 : 0; }
};
struct Product {
    LinPlan plan;
    Side a, b;
    size_t part, dpart;  // bytes
    size_t bytes() const { return a.bytes() + b.bytes() + part + dpart; }
};

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t over(int64_t v, int64_t by) { return (v + by - 1) / by; }

// Rows that fill a tile's 128 lanes no more than once go to its columns, and the other side to the lanes: twice as many tiles, each
// with as little of the rows as there is.  Likewise a k of at most 128 in the backward weight beside a wider n.
bool exchanged(int op, int64_t rows, int64_t k, int64_t n) { return op == OP_WGRAD ? k <= 128 && n > 128 : rows <= 128; }

// A way to cut a product, and about how long it takes.
struct Shape {
    bool pair;
    int bn, units, stage_bytes, split;
    int64_t tm, tn, whole, share;  // tiles dealt out whole; a unit's blocks of the others
    double ns;
};

// What a call's time is made of, in ns, as measured on its parts: 2000 until the first stage is there; a stage as its bytes come from
// L2 (105 a ns and SM, 118 at best) or its products run, whichever is longer; an epilogue of 1000 and 700 for each 128 columns, under
// the next tile's products if there is one; and where tiles are cut, writing parts at 50 bytes a ns and SM, and a second launch that
// reads them all at 4000.  A pair's launch and barriers take 700 more; over many rounds its tiles' epilogues go better (64 -> 256 on
// 2.1M rows 416 us on pairs, 562 on lone CTAs, whose stages are half as large again and only two fit).
bool shape(const LinGemm& G, bool pair, int bn, bool cut, Shape& t) {
    t.pair = pair, t.bn = bn;
    t.units = pair ? kPlanSms / 2 : kPlanSms;
    t.tm = over(G.m, pair ? 256 : 128), t.tn = over(G.n, bn);
    const int half = pair ? bn / 2 : bn;
    t.stage_bytes = (int)(16384 + (G.b_mn ? up(half, 64) * 128 : up(half * 128, 1024)));
    const double products = 4 / 1.9 * std::max(bn / 2.0, (4096 + 32.0 * bn) / 128), block = std::max(t.stage_bytes / 105.0, products);
    const double epilogue = 1000 + 700 * over(bn, 128), start = pair ? 2700 : 2000, round = pair ? epilogue : 1.3 * epilogue;
    const int64_t tiles = t.tm * t.tn, rounds = tiles / t.units, rem = tiles - rounds * t.units;
    t.whole = tiles, t.share = 1, t.split = 0;
    if (!cut) {
        const int64_t most = rounds + (rem > 0);
        t.ns = start + std::max(most * G.nkb * block, (most - 1) * round) + epilogue;
        return true;
    }
    t.whole = tiles - rem, t.share = std::max<int64_t>(2, over(rem * G.nkb, t.units));
    if (rem == 0 || t.share >= G.nkb) return false;
    const double bytes = 512.0 * bn, parts = over(rem * G.nkb, t.share) * (pair ? 2 : 1) * bytes;
    t.ns = start + std::max((rounds * G.nkb + t.share) * block, rounds * round) + 500 + bytes / 50 + 3000 + parts / 4000;
    return true;
}

// A tile to a cluster of `split` CTAs.  Clusters of four leave some of an SM group idle, so that about 128 CTAs run at a time.
// 2300 until the first stage is there; 2000, and 4 for each of a tile's columns, to add up; and the epilogue, which where rows are not on
// the columns goes by 32 columns with their loads' latency.
bool shape_split(const LinGemm& G, int op, bool swap, int bn, int split, Shape& t) {
    shape(G, false, bn, false, t);
    const int64_t tiles = t.tm * t.tn;
    if (split > G.nkb || tiles * split > (split > 2 ? 128 : 144)) return false;
    t.split = split;
    t.ns = 2300 + over(G.nkb, split) * std::max(t.stage_bytes / 105.0, 4 / 1.9 * std::max(bn / 2.0, (4096 + 32.0 * bn) / 128)) + 2000 + 4 * bn +
           (swap ? 500 : (op == OP_DGRAD ? 1000 : 600) * over(bn / split, 32));
    return true;
}

Product plan_of(const cf_linear_desc* d, int op) {
    const Side x{d->rows, d->k, x_pitch(d), op == OP_WGRAD}, w{d->n, d->k, d->k, op == OP_DGRAD}, dz{d->rows, d->n, y_pitch(d), op == OP_WGRAD};
    Product P{};
    LinGemm& G = P.plan.g;
    P.plan.swap = exchanged(op, d->rows, d->k, d->n);
    P.a = op == OP_FWD ? x : dz;
    P.b = op == OP_WGRAD ? x : w;
    G.m = op == OP_WGRAD ? d->n : d->rows;
    G.n = op == OP_FWD ? d->n : d->k;
    G.nkb = (int)over(op == OP_FWD ? d->k : op == OP_DGRAD ? d->n : d->rows, 64);
    if (P.plan.swap) std::swap(P.a, P.b), std::swap(G.m, G.n);
    G.a_mn = P.a.mn, G.b_mn = P.b.mn;

    // The tile and the cut that should be quickest.
    Shape best{}, t;
    for (const bool pair : {true, false}) {
        if (pair && (P.plan.swap || G.m <= 128 || G.n <= 128)) continue;
        for (const int at : {256, 192, 128, 64}) {
            if (P.plan.swap && at < 256) break;
            // the epilogue's passes of 64 columns end with a tile where another follows
            const int64_t tn = over(G.n, at);
            const int bn = (int)up(over(G.n, tn), tn > 1 ? 64 : pair ? 32 : 16);
            if (bn > 256) continue;
            for (const bool cut : {false, true})
                if (shape(G, pair, bn, cut, t) && (best.ns == 0 || t.ns < best.ns)) best = t;
            // of more blocks than the tensor cores may sum for an fp32 result there is no such kernel
            if (pair || op == OP_WGRAD) continue;
            for (const int split : {2, 4})
                if ((d->dtype != CF_DT_F32 || over(G.nkb, split) <= kMostSummed) && shape_split(G, op, P.plan.swap, bn, split, t) && t.ns < best.ns) best = t;
        }
    }
    P.plan.pair = best.pair;
    const int units = best.units;
    G.tm = (int)best.tm, G.tn = (int)best.tn, G.bn = best.bn;
    G.stage_bytes = best.stage_bytes;
    G.a_box = 128, G.b_box = best.pair ? best.bn / 2 : best.bn;
    // fp32 results of more blocks than the tensor cores may sum
    G.seg = kMostSummed;
    G.split = best.split;
    const int64_t most = std::max<int64_t>(best.whole ? G.nkb : 0, best.whole < best.tm * best.tn ? std::min<int64_t>(best.share, G.nkb) : 0);
    P.plan.sums = (op == OP_WGRAD || d->dtype == CF_DT_F32) && most > G.seg;
    // Narrow tiles of many rows: as many side by side as the accumulator holds, so that what a tile takes besides its products and
    // stores is taken less often; with rounds enough left to even out.
    G.sub = 1;
    if (!best.pair && !best.split && !P.plan.swap && !P.plan.sums && best.tn == 1 && best.whole == best.tm) {
        while (2 * G.sub * best.bn <= 256 && best.tm >= 8 * G.sub * best.units) G.sub *= 2;
        best.tm = over(G.m, 128 * G.sub), best.whole = best.tm;
        G.tm = (int)best.tm;
    }
    const int64_t tiles = best.tm * best.tn;
    G.whole = (int)best.whole, G.share = (int)best.share, G.rest = (tiles - best.whole) * G.nkb;
    const int64_t share = best.share;
    G.units = (int)(G.whole ? std::min<int64_t>(units, tiles) : over(G.rest, G.share));
    P.plan.cut = G.rest && share < G.nkb;
    if (P.plan.cut) {
        const size_t slots = 2 * (size_t)over(G.rest, G.share);
        P.part = slots * (P.plan.pair ? 2 : 1) * 128 * G.bn * sizeof(float);
        P.dpart = op == OP_WGRAD ? slots * 256 * sizeof(float) : 0;
    }
    return P;
}

cf_status pack(const LaunchCtx& ctx, const Side& s, const uint16_t*& at, char*& ws) {
    if (!s.packed()) return CF_OK;
    uint16_t* to = reinterpret_cast<uint16_t*>(ws);
    const int64_t blocks = std::min<int64_t>(over(s.rows * s.kept() / 8, 256), 16 * ctx.num_sms);
    linear_pack_kernel<<<(unsigned)blocks, 256, 0, ctx.stream>>>(at, s.rows, (int)s.width, s.pitch, to, (int)s.kept());
    at = to;
    ws += s.bytes();
    return status_of();
}
bool map_of(CUtensorMap* m, const Side& s, const uint16_t* at, int box) {
    const uint64_t dims[2] = {(uint64_t)s.width, (uint64_t)s.rows}, strides[1] = {(uint64_t)s.kept() * 2};
    const uint32_t boxes[2] = {64, (uint32_t)(s.mn ? 64 : box)};
    return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, at, dims, strides, boxes, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int OP>
cf_status product(const cf_linear_desc* d, const uint16_t* a, const uint16_t* b, LinEpi E, void* ws, size_t ws_bytes, void* stream) {
    Product P = plan_of(d, OP);
    if (P.bytes() && (ws == nullptr || ws_bytes < P.bytes())) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    if (P.plan.swap) std::swap(a, b);
    char* at = static_cast<char*>(ws);
    if (const cf_status st = pack(ctx, P.a, a, at); st != CF_OK) return st;
    if (const cf_status st = pack(ctx, P.b, b, at); st != CF_OK) return st;
    LinGemm& G = P.plan.g;
    const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    LinMaps M{};
    uint32_t room = kLinSmem - (uint32_t)sizeof(LinShared) - (OP == OP_WGRAD ? kLinOnes : 0);
    const bool sums = P.plan.sums, few = (int64_t)G.tm * G.tn <= 2 * G.units && G.bn > 128;
    LinStage& S = G.st;
    S.sets = few || sums ? 1 : 2, S.turns = few && !sums ? 4 : 2, S.gw = 32;
    if (!P.plan.swap && !G.split) {
        if (OP == OP_WGRAD && E.accumulate) E.add = E.out;
        const bool aux = E.pre_in || E.pre_out;
        S.load_add = E.add != nullptr, S.load_aux = E.pre_in != nullptr;
        // a stored row that ends inside 16 bytes would fill them up
        S.tma = E.pitch % 8 == 0 && E.cols % 8 == 0;
        S.gw = E.f32 && !aux ? 32 : 64;
        S.out_bytes = S.gw * (E.f32 ? 128 : 64), S.aux_bytes = aux ? 4096 : 0;
        // All warps, on one tile or on two in turn, where the epilogue is much of a tile's time and two stages fit beside their room;
        // else half of them, and more stages.
        const uint32_t pass = S.out_bytes + S.aux_bytes + (OP == OP_FWD ? kLinBias : 0);
        const bool all = !sums && G.nkb <= 16 && room >= kLinEpiWarps * pass + 2 * G.stage_bytes;
        S.sets = all && !few ? 2 : 1, S.turns = all && few ? 4 : 2;
        room -= 4 * S.sets * S.turns * pass;
        auto rows_map = [&](CUtensorMap* m, const void* p, bool f32) {
            const uint64_t dims[2] = {(uint64_t)E.cols, (uint64_t)E.rows}, strides[1] = {(uint64_t)E.pitch * (f32 ? 4 : 2)};
            const uint32_t box[2] = {f32 ? 32u : 64u, 32};
            return encode_tmap(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : bf16, 2, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        };
        const void* pre = OP == OP_FWD ? E.pre_out : E.pre_in;
        if (S.tma && (!rows_map(&M.out, E.out, E.f32) || (E.add && !rows_map(&M.add, E.add, E.f32)) || (aux && !rows_map(&M.aux, pre, false))))
            return CF_ERR_CUDA;
    }
    G.stages = std::min<int>(kLinMostStages, room / G.stage_bytes);
    G.part = reinterpret_cast<float*>(at);
    G.dpart = reinterpret_cast<float*>(at + P.part);
    G.status = ctx.status, G.wait_ns = ctx.wait_ns;
    if (!map_of(&M.a, P.a, a, G.a_box) || !map_of(&M.b, P.b, b, G.b_box)) return CF_ERR_CUDA;
    return launch_linear<OP>(ctx, P.plan, M, E);
}

__global__ void __launch_bounds__(256) linear_zero_kernel(float* p, int64_t count) {
    for (int64_t e = blockIdx.x * (int64_t)256 + threadIdx.x; e < count; e += (int64_t)gridDim.x * 256) p[e] = 0.f;
}

}  // namespace
}  // namespace cf

using namespace cf;

extern "C" {

size_t cf_linear_workspace_size(const cf_linear_desc* desc, int32_t op) {
    if (check(desc) != CF_OK || op < CF_LINEAR_FWD || op > CF_LINEAR_WGRAD || desc->rows == 0) return 0;
    return plan_of(desc, op).bytes();
}

cf_status cf_linear_fwd(const cf_linear_desc* desc, const uint16_t* x, const uint16_t* w, const float* bias, const void* residual, void* y,
                        uint16_t* pre, void* ws, size_t ws_bytes, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    if (desc->rows == 0) return CF_OK;
    if (!x || !w || !y) return CF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)x, (const void*)w, (const void*)bias, residual, (const void*)y, (const void*)pre, (const void*)ws})
        if (!aligned16(p)) return CF_ERR_INVALID_ARG;
    return product<OP_FWD>(desc, x, w,
                           LinEpi{bias, residual, nullptr, pre, y, nullptr, y_pitch(desc), desc->rows, desc->n, desc->act, desc->dtype == CF_DT_F32, 0,
                                  desc->slope, desc->scale},
                           ws, ws_bytes, stream);
}

cf_status cf_linear_act_bwd(const cf_linear_desc* desc, const void* dy, const uint16_t* pre, uint16_t* dz, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    if (desc->rows == 0) return CF_OK;
    if (!dy || !pre || !dz || !aligned16(dy) || !aligned16(pre) || !aligned16(dz)) return CF_ERR_INVALID_ARG;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    LinEpi E{};
    E.act = desc->act, E.f32 = desc->dtype == CF_DT_F32, E.slope = desc->slope, E.scale = desc->scale;
    const int64_t pitch = y_pitch(desc), blocks = std::min<int64_t>(over(desc->rows * over(desc->n, 8), 256), 16 * ctx.num_sms);
    auto kernel = desc->n % 8 == 0 && pitch % 8 == 0 ? linear_act_bwd_kernel<true> : linear_act_bwd_kernel<false>;
    kernel<<<(unsigned)blocks, 256, 0, ctx.stream>>>(dy, pre, dz, desc->rows, desc->n, pitch, E);
    return status_of();
}

cf_status cf_linear_dgrad(const cf_linear_desc* desc, const uint16_t* dz, const uint16_t* w, const uint16_t* pre, const void* add, void* dx,
                          void* ws, size_t ws_bytes, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    if (desc->rows == 0) return CF_OK;
    if (!dz || !w || !dx) return CF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)dz, (const void*)w, (const void*)pre, add, (const void*)dx, (const void*)ws})
        if (!aligned16(p)) return CF_ERR_INVALID_ARG;
    return product<OP_DGRAD>(desc, dz, w,
                             LinEpi{nullptr, add, pre, nullptr, dx, nullptr, x_pitch(desc), desc->rows, desc->k, desc->act, desc->dtype == CF_DT_F32,
                                    0, desc->slope, desc->scale},
                             ws, ws_bytes, stream);
}

cf_status cf_linear_wgrad(const cf_linear_desc* desc, const uint16_t* x, const uint16_t* dz, float* dw, float* db, int32_t accumulate, void* ws,
                          size_t ws_bytes, void* stream) {
    if (const cf_status st = check(desc); st != CF_OK) return st;
    if ((desc->rows && (!x || !dz)) || !dw) return CF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)x, (const void*)dz, (const void*)dw, (const void*)db, (const void*)ws})
        if (!aligned16(p)) return CF_ERR_INVALID_ARG;
    if (desc->rows == 0) {
        LaunchCtx ctx;
        if (accumulate) return CF_OK;
        if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
        const int64_t count = (int64_t)desc->n * desc->k;
        linear_zero_kernel<<<(unsigned)std::min<int64_t>(over(count, 256), 16 * ctx.num_sms), 256, 0, ctx.stream>>>(dw, count);
        if (const cf_status st = status_of(); st != CF_OK || !db) return st;
        linear_zero_kernel<<<(unsigned)std::min<int64_t>(over(desc->n, 256), 16 * ctx.num_sms), 256, 0, ctx.stream>>>(db, desc->n);
        return status_of();
    }
    return product<OP_WGRAD>(desc, dz, x,
                             LinEpi{nullptr, nullptr, nullptr, nullptr, dw, db, desc->k, desc->n, desc->k, CF_ACT_LRELU, 1, accumulate != 0, 1.f,
                                    desc->scale},
                             ws, ws_bytes, stream);
}

}  // extern "C"
