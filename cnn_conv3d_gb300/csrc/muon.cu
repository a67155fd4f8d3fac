// muon.cu -- orthogonalisation of matrices by Newton-Schulz products and the
// momentum step that uses it, with their entry points.
//
// Of k x n values, k <= n, matrices of a call that all have at most 32 rows go to ns_tiny_kernel, all of at most 128 to
// ns_small_kernel, each up to a length (tiny_of, cluster_of); the others take three launches for all of a call, but for those of few
// values, which ns_tiny_kernel takes out of any list (take_few).  ns_input_kernel
// takes the momentum step and the Frobenius norms' partial sums, ns_convert_kernel writes X = u / (|u| + eps) in operand form, and
// ns_kernel is one cooperative launch of a CTA per SM that runs the steps as phases between grid-wide barriers; a phase's
// items (tiles of all matrices) are dealt out over the CTAs, or over pairs of them:
//   G  A' = X X^T - alpha I (tiles on and above the diagonal), or parts of the sums where the CTAs take even shares of all
//      tiles' blocks
//   R  A' from the parts, where there are any
//   S  B' = (b + 2 c alpha) A' + c A' A'     (so b A + c A^2 = beta I + B',
//                                             beta = b alpha + c alpha^2)
//   U  X = a X + beta X + B' X; the last step writes the result instead
//
// Operands are fp16 (11 bits; bf16's 8 gave 1e-2 to 3e-1), sums fp32, and X has a byte a value beside its operand (rest_of).
// Near the end A is close to I: taking alpha and beta off before rounding keeps the rounding relative to what is left.  Of
// beta X, the last two steps take X and the earlier ones its operand: there B' X cancels beta X along directions whose
// singular value is still small, and has the operand only.
// Any alpha gives the same polynomial; it is where a flat spectrum would be, a^(2 step) / k, up to the value that the
// polynomial leaves in place.  Simulated against 64 bits (operands rounded, sums exact): 3e-4 to 1.2e-3 of the result, where
// rounding A and B with their diagonals gives up to 4e-3, and the mean of A's diagonal for alpha 2e-4 to 1e-3.  Measured:
// 1.1e-3 for 2048 x 8192, 1.4e-3 for 1511 x 515, both before the result's rounding to bf16.
// X is scaled by a power of two tau so that its entries stay well inside
// fp16's normal range for every size.
//
// Operands live in blocks of 64 x 64 in the order that the tensor cores read
// from shared memory (128-byte rows, 16-byte chunks XORed by the row), zero
// where a matrix ends inside a block, so that a tile is fetched by bulk copies
// without a tensor map and nothing has to be masked.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <new>
#include <vector>

#include "cf_internal.h"
#include "cf_ptx.cuh"

namespace cf {
namespace {

constexpr int kNormChunks = 1024;         // partial sums of a matrix's norm, at most
constexpr float kDown = 0x1p-80f;         // scale of the sums that stand in for overflowing ones
constexpr float kUp = 0x1p100f, kLow = 0x1p-100f;  // scale of those for sums below kLow, of whose squares some or all are lost
constexpr int kMaxMats = 48;              // matrices of one launch
constexpr int kEpiWarps = 12;             // epilogue warps
constexpr int kThreads = 64 + 32 * kEpiWarps;  // producer, issuer, epilogue
constexpr int kBlk = 64 * 64;             // values of an operand block
constexpr uint32_t kBlkBytes = kBlk * 2;
constexpr uint32_t kRing = 24 * kBlkBytes;  // operand stages: as many as fit, of 4 or 6 blocks
constexpr int kMostStages = 6;
constexpr uint32_t kSmem = kRing + 1024;
constexpr int kTileF = 128 * 128;         // floats of a Gram tile

constexpr int kPlanSms = 152;             // SMs that work is planned for: workspaces are laid out without asking the device

struct Mat {
    const void* g;
    float* m;
    float* w;
    uint16_t* o;
    int64_t rows, cols;      // as stored
    int k, n;                // k <= n; transposed when rows > cols
    int f32, tall;
    float keep, step;        // w = keep w - step X
    float tau;
    int vec, wide;           // rows start at 16 bytes, those of the result at 32
    int aligned;             // g starts at 16 bytes
    int rb, cb, nx;          // operand blocks: X is rb x cb, of which nx have columns, A' and B' rb x rb
    int mt, gt, ut;          // 128-row tiles, rows of tiles (1, in pairs 2, of those each), columns of tiles of phase U
    int chunks;              // norm partials
    int64_t chunk;           // values of each
    int n0, c0, s0, u0;      // first item of each phase
    int b0;                  // first block of phase G
    __half *xh[2], *ad, *bp;
    uint8_t* x;              // the bytes that X has more than its operand
    float *d, *norm;
};

// A tile of the Gram matrix whose long axis is cut: the unit that makes its first part, and how many units make one.
struct Cut {
    int16_t mat, i, j;
    uint8_t unit, parts;
};

struct Job {
    Mat mat[kMaxMats];
    Cut cut[kPlanSms];
    int count, steps;
    int nn, nc, ns, nu;  // items of each phase; G has S's
    int share, blocks;   // phase G cut into shares of so many blocks of all its tiles' (0: whole tiles)
    int cuts;
    int half_g, half;    // G (where it is not cut) and S in tiles of half the columns
    int uw;              // 64-column blocks of a tile of U
    int whole;           // tiles of U before those that are taken in halves
    float* part;
    float a, b, c, eps, mu, cap;
    int nesterov;
    uint32_t* sync;  // arrivals at the grid barrier, abort flag
    int* status;
    uint64_t wait_ns;
};

// The three sums of squares of a matrix's values.
__device__ __forceinline__ void add_squares(float u, float& s, float& down, float& up) {
    const float d = u * kDown, p = u * kUp;
    s = fmaf(u, u, s);
    down = fmaf(d, d, down);
    up = fmaf(p, p, up);
}
// Which of the three sums gives the norm: 0, 1 (down), 2 (up; beside an eps of 1 or more the values are nothing).
__device__ __forceinline__ int which_sum(float s, float eps) { return isinf(s) ? 1 : s < kLow && eps < 1.f ? 2 : 0; }
// tau u / (|u| + eps) as (u pre) inv, from the sum that which_sum names; a zero matrix gives zero whatever eps is.
__device__ __forceinline__ void scale_of(int which, float sum, float eps, float tau, float& pre, float& inv) {
    pre = which == 1 ? kDown : which == 2 ? kUp : 1.f;
    const float den = sqrtf(sum) + eps * pre;
    inv = den == 0.f ? 0.f : tau / den;
}

// A launch that is enqueued under the end of one of its list's small matrices, which it has nothing to do with, still ends after it.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float load_u(const Mat& M, const Job& J, int64_t i) {
    float u = M.f32 ? static_cast<const float*>(M.g)[i] : bf16_bits_to_float(static_cast<const uint16_t*>(M.g)[i]);
    if (M.m) u = J.nesterov ? fmaf(J.mu, M.m[i], u) : M.m[i];
    return u;
}

// Memory bounds this pass: 2048 x 8192 fp32 in 16 us, 4.0 TB/s, the seven convolutions' g and m (76 MB) in 18 us, 4.3 TB/s and the
// writes.  256 blocks a matrix and a value a load took 110 us with the next pass, 1024 blocks and four values 48.
// The momentum step of one chunk, and its sums of u^2, of (kDown u)^2, which stands in where the first overflows, and of (kUp u)^2,
// which does where it underflows.
__global__ void __launch_bounds__(256) ns_input_kernel(const __grid_constant__ Job J) {
    __shared__ float red[24];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x < 2) J.sync[threadIdx.x] = 0;
    int i = 0;
    while (i + 1 < J.count && (int)blockIdx.x >= J.mat[i + 1].n0) ++i;
    const Mat& M = J.mat[i];
    int64_t b = (blockIdx.x - M.n0) * M.chunk;
    const int64_t e = min(b + M.chunk, M.rows * M.cols);
    float s = 0.f, s2 = 0.f, s3 = 0.f;
    auto one = [&](float u, float m, float& mo) {  // mo: m's successor
        if (M.m) {
            mo = fmaf(J.mu, m, u);
            u = J.nesterov ? fmaf(J.mu, mo, u) : mo;
        }
        add_squares(u, s, s2, s3);
    };
    if (M.f32 && M.aligned) {
        // chunks are whole vectors but for the matrix's end
        const int64_t e4 = b + (e - b) / 4 * 4;
#pragma unroll 2
        for (int64_t j = b + 4 * threadIdx.x; j < e4; j += 1024) {
            const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(M.g) + j);
            float4 m = M.m ? *reinterpret_cast<const float4*>(M.m + j) : make_float4(0.f, 0.f, 0.f, 0.f);
            one(u.x, m.x, m.x);
            one(u.y, m.y, m.y);
            one(u.z, m.z, m.z);
            one(u.w, m.w, m.w);
            if (M.m) *reinterpret_cast<float4*>(M.m + j) = m;
        }
        b = e4;
    }
#pragma unroll 4
    for (int64_t j = b + threadIdx.x; j < e; j += 256) {
        const float u = M.f32 ? static_cast<const float*>(M.g)[j] : bf16_bits_to_float(static_cast<const uint16_t*>(M.g)[j]);
        float m = M.m ? M.m[j] : 0.f;
        one(u, m, m);
        if (M.m) M.m[j] = m;
    }
    for (int o = 16; o; o >>= 1) {
        s += __shfl_down_sync(~0u, s, o);
        s2 += __shfl_down_sync(~0u, s2, o);
        s3 += __shfl_down_sync(~0u, s3, o);
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s, red[8 + (threadIdx.x >> 5)] = s2, red[16 + (threadIdx.x >> 5)] = s3;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int t = 1; t < 8; ++t) s += red[t], s2 += red[8 + t], s3 += red[16 + t];
        M.norm[blockIdx.x - M.n0] = s;
        M.norm[kNormChunks + blockIdx.x - M.n0] = s2;
        M.norm[2 * kNormChunks + blockIdx.x - M.n0] = s3;
        after_previous();
    }
}

// Sum of v[0 .. count) over a block of 256 threads, the same everywhere and in a fixed order; all threads call it.
__device__ __forceinline__ float block_sum(const float* v, int count, float* red) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kNormChunks / 256; ++i)
        if ((int)threadIdx.x + 256 * i < count) s += v[threadIdx.x + 256 * i];
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
    for (int i = 0; i < 8; ++i) s += red[i];
    return s;
}

// alpha of a step: where a flat spectrum's squared singular values would be, at most what the polynomial leaves in place.
__device__ __forceinline__ float alpha_of(float a, float cap, int k, int step) {
    float t = 1.f / (float)k;
    for (int i = 0; i < step; ++i) t *= a * a;
    return fminf(t, cap);
}

// Offset in values of element (r, c) of a blocked operand with cb blocks a row.
__device__ __forceinline__ int64_t blocked(int r, int c, int cb) {
    return ((int64_t)(r >> 6) * cb + (c >> 6)) * kBlk + (r & 63) * 64 + ((((c & 63) >> 3) ^ (r & 7)) << 3) + (c & 7);
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// fp16 operands, fp32 sums: M x N, A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

struct Shared {
    uint64_t full[kMostStages], empty[kMostStages], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int abort;
};

// All CTAs of the grid: what any of them wrote before is seen by all after, by bulk copies too.  One thread's fences stand for
// the block's: its barriers order them after, and before, everyone's accesses.
__device__ bool grid_sync(const Job& J, uint32_t& target, Shared& sh) {
    __syncthreads();
    if (threadIdx.x == 0) {
        target += gridDim.x;
        if (*(volatile int*)&sh.abort) atomicExch(&J.sync[1], 1u);
        fence_async();
        asm volatile("red.release.gpu.add.u32 [%0], 1;" ::"l"(&J.sync[0]) : "memory");
        const uint64_t t0 = globaltimer();
        uint32_t seen, stop = 0;
        while (true) {
            asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(seen) : "l"(&J.sync[0]) : "memory");
            if (seen >= target) break;
            if (globaltimer() - t0 < 50000) continue;  // the abort flag is for waits that are already long
            asm volatile("ld.relaxed.gpu.u32 %0, [%1];" : "=r"(stop) : "l"(&J.sync[1]) : "memory");
            if (stop == 0 && globaltimer() - t0 > J.wait_ns) {
                atomicCAS(J.status, 0, (int)WAIT_GRID);
                atomicExch(&J.sync[1], 1u);
                stop = 1;
            }
            if (stop) break;
        }
        if (stop) sh.abort = 1;
        fence_async();
    }
    __syncthreads();
    return sh.abort == 0;
}

enum { PH_G, PH_S, PH_U };

// The products run on single CTAs, a tile of 128 rows each, or (PAIR) on pairs that share one of 256 rows: each CTA fetches its
// own half of the rows and of the other side, and one instruction multiplies for both.  A pair's stages hold half as much for
// the same products, so that twice as many are in flight.
template <bool PAIR>
__device__ __forceinline__ int unit_id() { return PAIR ? blockIdx.x >> 1 : blockIdx.x; }
template <bool PAIR>
__device__ __forceinline__ int unit_count() { return PAIR ? gridDim.x >> 1 : gridDim.x; }

// An item of a product phase: which operand blocks, and how many.
struct Item {
    int mat, i, j;  // tile, tile of the other side
    int kb0, kb1;   // blocks of the contracted axis
    int cb0;        // its first 64-column block (S: within the tile of the other side)
    int nb;         // 64-column blocks of the item
    int slot;       // where a part of a tile goes, -1 for a whole one
};

// Tile e of those on and above the diagonal of t x t tiles, row by row.
__device__ __forceinline__ void upper_tile(int e, int t, int& i, int& j) {
    i = 0;
    while (e >= t - i) {
        e -= t - i;
        ++i;
    }
    j = i + e;
}

// A unit's way through a phase: items in turn, or in phase G, where it is cut, the tiles of an even share of all blocks.  A share
// has at most two parts of tiles, one that its tile's other parts come before (the slot 2 unit) and one that they come after.
template <int PH, bool PAIR>
struct Walk {
    int it, at = 0, end = 0, mat = 0;
    __device__ __forceinline__ Walk() : it(unit_id<PAIR>()) {}
    __device__ __forceinline__ bool next(const Job& J, Item& t) {
        t.kb0 = 0, t.slot = -1, t.cb0 = 0, t.nb = PAIR ? 4 : 2;
        int e;
        if (PH == PH_G && J.share) {
            if (at == end) {
                at = it * J.share, end = min(at + J.share, J.blocks);
                if (at >= J.blocks) return false;
                it += unit_count<PAIR>();
            }
            while (mat + 1 < J.count && at >= J.mat[mat + 1].b0) ++mat;
            const Mat& M = J.mat[mat];
            e = (at - M.b0) / M.nx;
            t.kb0 = (at - M.b0) - e * M.nx;
            t.kb1 = min(M.nx, t.kb0 + end - at);
            at += t.kb1 - t.kb0;
            if (t.kb1 - t.kb0 < M.nx) t.slot = 2 * (it - unit_count<PAIR>()) + (t.kb0 == 0);
        } else {
            const bool half = PH == PH_G ? J.half_g : PH == PH_S ? J.half : PH == PH_U && PAIR && it >= J.whole;
            const int from = PH == PH_U ? J.whole : 0, which = half ? (it - from) & 1 : 0;
            const int at = half ? from + ((it - from) >> 1) : it;
            if (at >= (PH == PH_U ? J.nu : J.ns)) return false;
            while (mat + 1 < J.count && at >= (PH == PH_U ? J.mat[mat + 1].u0 : J.mat[mat + 1].s0)) ++mat;
            const Mat& M = J.mat[mat];
            e = at - (PH == PH_U ? M.u0 : M.s0);
            t.nb = (PAIR ? 4 : 2) >> half;
            t.cb0 = which * t.nb;
            t.kb1 = PH == PH_G ? M.nx : (M.k + 63) / 64;
            it += unit_count<PAIR>();
        }
        const Mat& M = J.mat[mat];
        t.mat = mat;
        if (PH == PH_U) {
            t.i = e % M.gt;
            t.j = e / M.gt;
            t.cb0 += J.uw * t.j;
            if (!PAIR) t.nb = min(J.uw, M.cb - t.cb0);
        } else {
            upper_tile(e, M.gt, t.i, t.j);
        }
        return true;
    }
};

// A role's way through the ring: each stage's parity, kept over phases that cut the ring differently.
struct Pipe {
    int stage = 0;
    uint32_t bits = 0, local = 0;
    uint32_t issued = 0;  // stages that a copy was issued for
    __device__ __forceinline__ uint32_t parity() const { return (bits >> stage) & 1; }
    __device__ __forceinline__ void next(int stages) {
        bits ^= 1u << stage;
        if (++stage == stages) stage = 0;
    }
};
// Whether the other side's rows are the tile's, in shared memory at the same place.
template <int PH, bool PAIR>
__device__ __forceinline__ bool same_side(const Item& t) { return PH != PH_U && t.i == t.j && !(PAIR && t.nb < 4); }

// Blocks of a stage in a phase: two of the CTA's rows, and the other side's.
template <int PH, bool PAIR>
__device__ __forceinline__ int stage_blocks(const Job& J) { return PH == PH_U && !PAIR && J.uw > 2 ? 6 : 4; }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* at, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    return a;
}
// An arrival at the first CTA's barrier, from either CTA of a pair.  What it announces is in place by then for every reader
// (copies that have landed in shared memory, tensor memory that has been read): it orders no accesses of its own, and a release
// for the cluster took the products from 0.25 to 0.7 us a stage.
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote(bar, 0)) : "memory");
}
// D (both CTAs' tensor memory) (+)= A B: 256 rows, each CTA's shared memory holding half of A's and of B's rows at the same place.
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives at both CTAs' barrier when the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

// A warp: each lane issues its own copy of a stage (one thread issuing eight took 1.4 us a stage).
template <int PH, bool PAIR>
__device__ __forceinline__ void produce(const Job& J, int cur, Shared& sh, uint8_t* ring, Pipe& P) {
    const int lane = threadIdx.x & 31, rank = PAIR ? (int)cluster_rank() : 0;
    const int sb = stage_blocks<PH, PAIR>(J), stages = 24 / sb;
    P.stage = 0;
    Walk<PH, PAIR> way;
    Item t;
    while (way.next(J, t)) {
        const Mat& M = J.mat[t.mat];
        const __half* a = PH == PH_G ? M.xh[cur] : PH == PH_S ? M.ad : M.bp;
        const int acb = PH == PH_G ? M.cb : M.rb;
        const bool same = same_side<PH, PAIR>(t);
        const int cols = PAIR ? t.nb / 2 : t.nb;  // blocks of the other side that the CTA fetches
        const uint32_t bytes = (2 + (same ? 0 : cols)) * kBlkBytes;
        // the lane's copy of each stage: a block of the tile's rows (lanes 0, 1), of the other side's rows (2, 3), or (U, lane 2)
        // X's row of blocks
        const bool isb = lane >= 2, row = PH == PH_U && isb;
        const int q = lane & 1;
        const bool mine = lane < 2 || (!same && lane < (PH == PH_U ? 3 : 2 + cols));
        const int tr = (PAIR ? 4 : 2) * (isb ? t.j : t.i) + (isb ? t.cb0 + cols * rank : 2 * rank) + q;
        const __half* src = row ? M.xh[cur] + ((int64_t)t.kb0 * M.cb + t.cb0 + cols * rank) * kBlk : a + ((int64_t)tr * acb + t.kb0) * kBlk;
        const int64_t step = row ? (int64_t)M.cb * kBlk : kBlk;
        const uint32_t size = row ? cols * kBlkBytes : kBlkBytes, dst = (isb ? 2 + (row ? 0 : q) : q) * kBlkBytes;
        for (int kb = t.kb0; kb < t.kb1; ++kb, src += step) {
            const bool ok = mbar_wait(&sh.empty[P.stage], P.parity() ^ 1, &sh.abort, J.wait_ns, J.status, WAIT_PRODUCER_EMPTY);
            if (!__all_sync(~0u, ok)) return;
            uint64_t* bar = &sh.full[P.stage];
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (mine) bulk_load(ring + P.stage * sb * kBlkBytes + dst, src, size, bar);
            P.issued |= 1u << P.stage;
            P.next(stages);
        }
    }
}

// One thread.  In a pair the first CTA's issues for both; the second's tells it of each of its own stages that is full.
template <int PH, bool PAIR>
__device__ __forceinline__ void issue(const Job& J, Shared& sh, uint8_t* ring, Pipe& P) {
    const int sb = stage_blocks<PH, PAIR>(J), stages = 24 / sb;
    const bool second = PAIR && cluster_rank() == 1;
    P.stage = 0;
    Walk<PH, PAIR> way;
    Item t;
    for (; way.next(J, t); ++P.local) {
        if (second) {
            for (int kb = t.kb0; kb < t.kb1; ++kb) {
                if (!mbar_wait(&sh.full[P.stage], P.parity(), &sh.abort, J.wait_ns, J.status, WAIT_MMA_FULL)) return;
                arrive_first(&sh.full[P.stage]);
                P.next(stages);
            }
            continue;
        }
        const uint32_t acc = P.local & 1, use = P.local >> 1, d = sh.tmem + acc * 256;
        if (!mbar_wait(&sh.tempty[acc], (use & 1) ^ 1, &sh.abort, J.wait_ns, J.status, WAIT_MMA_TMEM_EMPTY)) return;
        tc_fence_after();
        const bool same = same_side<PH, PAIR>(t);
        const uint32_t idesc = idesc_f16(PAIR ? 256 : 128, 64 * t.nb, PH == PH_U);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
            if (!mbar_wait(&sh.full[P.stage], P.parity(), &sh.abort, J.wait_ns, J.status, WAIT_MMA_FULL)) return;
            tc_fence_after();
            const uint32_t as = smem_u32(ring + P.stage * sb * kBlkBytes), bs = as + (same ? t.cb0 : 2) * kBlkBytes;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint64_t ad = sdesc(as + k * 32, 16, 1024, SWZ_128B);
                // X as [contracted][columns]: 64-column atoms a block apart, 16 contracted rows a step
                const uint64_t bd = PH == PH_U ? sdesc(bs + k * 2048, kBlkBytes, 1024, SWZ_128B)
                                               : sdesc(bs + k * 32, 16, 1024, SWZ_128B);
                if (PAIR)
                    umma_pair(d, ad, bd, idesc, kb > t.kb0 || k > 0);
                else
                    umma_bf16(d, ad, bd, idesc, kb > t.kb0 || k > 0);
            }
            if (PAIR)
                commit_pair(&sh.empty[P.stage]);
            else
                umma_commit(&sh.empty[P.stage]);
            P.next(stages);
        }
        if (PAIR)
            commit_pair(&sh.tfull[acc]);
        else
            umma_commit(&sh.tfull[acc]);
    }
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Columns c .. c+3 of row r of a 128-row tile in fp32: four columns of all rows in turn, so that lanes that own rows (as
// tensor memory is read) access consecutive 16 bytes.
__device__ __forceinline__ float4* tile_at(float* tile, int r, int c) {
    return reinterpret_cast<float4*>(tile) + (c >> 2) * 128 + r;
}

// X beside its operand: a byte a value (24 bits in all in place of 32, the products' operands having 11: against fp32 the result
// is as far from 64 bits as before, 1.1e-3 to 1.4e-3, and five steps of 2048 x 8192 went from 600 to 565 us), (x - h) / (2^-18 e) + 128 with h the operand's value and e the power of two in it, so
// that the two hold x to 2^-20 of it; a quarter of fp32's bytes, and with the operand, that is read and written anyway, three
// fifths of the traffic of phase U that X in fp32 took.  16 bytes of a row are together, then those of the tile's next row.
__device__ __forceinline__ uint4* rest_at(const Mat& M, int i, int j) {
    return reinterpret_cast<uint4*>(M.x + (int64_t)(i >> 7) * M.cb * 64 * 128) + (j >> 4) * 128 + (i & 127);
}
__device__ __forceinline__ float power_of(float h) {
    return fmaxf(__uint_as_float(__float_as_uint(h) & 0x7F800000u), 0x1p-14f);  // fp16's smallest normal value
}
__device__ __forceinline__ uint32_t rest_of(float x, float h) {
    const float inv = __uint_as_float(0x7F000000u - __float_as_uint(power_of(h)));
    return __float_as_uint(fminf(fmaf((x - h) * inv, 0x1p18f, 0x1p23f + 128.f), 0x1p23f + 255.f));  // in the lowest byte
}
__device__ __forceinline__ uint32_t pack_rest4(const float* x, const float* h) {
    const uint32_t lo = __byte_perm(rest_of(x[0], h[0]), rest_of(x[1], h[1]), 0x0040);
    const uint32_t hi = __byte_perm(rest_of(x[2], h[2]), rest_of(x[3], h[3]), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
// Value e of four: 32 + byte 2^-18 as a float, from which 32 and the bias are taken.
__device__ __forceinline__ float with_rest(float h, uint32_t bytes, int e) {
    const float d = __uint_as_float(__byte_perm(bytes, 0x42000000u, 0x7650 | e)) - (32.f + 128.f * 0x1p-18f);
    return fmaf(d, power_of(h), h);
}
__device__ __forceinline__ void unpack2_f16(uint32_t v, float& a, float& b) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
    a = f.x, b = f.y;
}

struct StepScalars {
    float alpha, beta, theta;  // theta: the part of beta that takes X in fp32
};
__device__ __forceinline__ StepScalars scalars_of(const Job& J, const Mat& M, int step) {
    StepScalars s;
    s.alpha = alpha_of(J.a, J.cap, M.k, step);
    s.beta = s.alpha * fmaf(J.c, s.alpha, J.b);
    s.theta = step + 2 >= J.steps ? s.beta : 0.f;
    return s;
}

__device__ __forceinline__ uint4 pack8_f16(const float* y) {
    return make_uint4(pack_f16(y[0], y[1]), pack_f16(y[2], y[3]), pack_f16(y[4], y[5]), pack_f16(y[6], y[7]));
}
// 16 values of row i, columns j .. j+15, into or from a blocked operand: a 32-byte access to two chunks, which the XOR keeps side
// by side.
__device__ __forceinline__ void store_row16(__half* op, int i, int j, int cb, uint4 p, uint4 q) {
    if (i & 1) {
        const uint4 t = p;
        p = q;
        q = t;
    }
    __half* at = op + (blocked(i, j, cb) & ~(int64_t)15);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(p.x), "r"(p.y), "r"(p.z), "r"(p.w),
                 "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w)
                 : "memory");
}
__device__ __forceinline__ void store_row16(__half* op, int i, int j, int cb, const float* y) {
    store_row16(op, i, j, cb, pack8_f16(y), pack8_f16(y + 8));
}
__device__ __forceinline__ void load_row16(const __half* op, int i, int j, int cb, uint32_t (&w)[8]) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(op + (blocked(i, j, cb) & ~(int64_t)15)));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) { return pack_bf16x2(a, b); }

// The result at row i, columns j .. j+C-1, from the last iterate (scaled by tau); the matrix starts `off` values on.
template <int C>
__device__ __forceinline__ void write_result(const Mat& M, int64_t off, int i, int j, float (&y)[C]) {
    const float inv = 1.f / M.tau;
    const int cnt = min(C, M.n - j);
    if (cnt <= 0) return;
    if (M.wide && cnt == C) {
        // lanes' rows lie apart, so that an access of 32 bytes a lane takes no longer than one of 16
        const int64_t base = off + (int64_t)i * M.n + j;
        if (M.w) {
            float w[C];
#pragma unroll
            for (int e = 0; e < C; e += 8)
                asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=f"(w[e]), "=f"(w[e + 1]), "=f"(w[e + 2]), "=f"(w[e + 3]), "=f"(w[e + 4]), "=f"(w[e + 5]),
                               "=f"(w[e + 6]), "=f"(w[e + 7])
                             : "l"(M.w + base + e));
#pragma unroll
            for (int e = 0; e < C; ++e) y[e] = M.keep * w[e] - M.step * (y[e] * inv);
#pragma unroll
            for (int e = 0; e < C; e += 8)
                asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(M.w + base + e), "f"(y[e]),
                             "f"(y[e + 1]), "f"(y[e + 2]), "f"(y[e + 3]), "f"(y[e + 4]), "f"(y[e + 5]), "f"(y[e + 6]),
                             "f"(y[e + 7])
                             : "memory");
        } else {
#pragma unroll
            for (int e = 0; e < C; ++e) y[e] *= inv;
        }
        if (M.o) {
#pragma unroll
            for (int e = 0; e < C; e += 16)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(M.o + base + e),
                             "r"(pack_bf16(y[e], y[e + 1])), "r"(pack_bf16(y[e + 2], y[e + 3])),
                             "r"(pack_bf16(y[e + 4], y[e + 5])), "r"(pack_bf16(y[e + 6], y[e + 7])),
                             "r"(pack_bf16(y[e + 8], y[e + 9])), "r"(pack_bf16(y[e + 10], y[e + 11])),
                             "r"(pack_bf16(y[e + 12], y[e + 13])), "r"(pack_bf16(y[e + 14], y[e + 15]))
                             : "memory");
        }
        return;
    }
    if (M.vec && cnt == C) {
        const int64_t base = off + (int64_t)i * M.n + j;
        if (M.w) {
            float4 w[C / 4];
#pragma unroll
            for (int e = 0; e < C / 4; ++e) w[e] = *reinterpret_cast<const float4*>(M.w + base + 4 * e);
#pragma unroll
            for (int e = 0; e < C / 4; ++e) {
                w[e].x = y[4 * e] = M.keep * w[e].x - M.step * (y[4 * e] * inv);
                w[e].y = y[4 * e + 1] = M.keep * w[e].y - M.step * (y[4 * e + 1] * inv);
                w[e].z = y[4 * e + 2] = M.keep * w[e].z - M.step * (y[4 * e + 2] * inv);
                w[e].w = y[4 * e + 3] = M.keep * w[e].w - M.step * (y[4 * e + 3] * inv);
                *reinterpret_cast<float4*>(M.w + base + 4 * e) = w[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < C; ++e) y[e] *= inv;
        }
        if (M.o) {
#pragma unroll
            for (int e = 0; e < C; e += 8)
                *reinterpret_cast<uint4*>(M.o + base + e) =
                    make_uint4(pack_bf16(y[e], y[e + 1]), pack_bf16(y[e + 2], y[e + 3]), pack_bf16(y[e + 4], y[e + 5]),
                               pack_bf16(y[e + 6], y[e + 7]));
        }
        return;
    }
    // transposed: the lanes' rows are consecutive values; else a ragged end or rows that start anywhere
    const int64_t base = off + (M.tall ? (int64_t)j * M.k + i : (int64_t)i * M.n + j), st = M.tall ? M.k : 1;
    if (M.w) {
        float w[C];
#pragma unroll
        for (int e = 0; e < C; ++e) w[e] = e < cnt ? M.w[base + e * st] : 0.f;
#pragma unroll
        for (int e = 0; e < C; ++e) {
            y[e] = M.keep * w[e] - M.step * (y[e] * inv);
            if (e < cnt) M.w[base + e * st] = y[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < C; ++e) y[e] *= inv;
    }
    if (M.o) {
#pragma unroll
        for (int e = 0; e < C; ++e)
            if (e < cnt) M.o[base + e * st] = __bfloat16_as_ushort(__float2bfloat16_rn(y[e]));
    }
}

// A' at row i, columns j .. j+15 of the tile d (in fp32): kept in fp32 and as an operand, on both sides of the diagonal.
__device__ __forceinline__ void store_gram16(const Mat& M, float* d, int r, int c, int i, int j, bool mirror, const float (&o)[16]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) *tile_at(d, r, c + 4 * e) = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
    store_row16(M.ad, i, j, M.rb, o);
    if (mirror) {
#pragma unroll
        for (int e = 0; e < 16; ++e) M.ad[blocked(j + e, i, M.rb)] = __float2half_rn(o[e]);
    }
}
// The 128 x 128 tile (ti, tj), ti <= tj, of A' in fp32.
__device__ __forceinline__ float* gram_tile(const Mat& M, int ti, int tj) {
    return M.d + (int64_t)(ti * M.mt - ti * (ti - 1) / 2 + tj - ti) * kTileF;
}

// 16 columns of the thread's row at a time, the warps of a row quarter in turn.
template <int PH, bool PAIR>
__device__ __forceinline__ void epilogue(const Job& J, int cur, int step, Shared& sh, Pipe& P) {
    constexpr int kTurn = kEpiWarps / 4, kTile = PAIR ? 2 : 1;  // 128-row tiles of a tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, turn = (warp - 2) >> 2;
    const int r = 32 * q + lane, rank = PAIR ? (int)cluster_rank() : 0;
    Walk<PH, PAIR> way;
    Item t;
    for (; way.next(J, t); ++P.local) {
        const Mat& M = J.mat[t.mat];
        const StepScalars sc = scalars_of(J, M, step);
        const uint32_t acc = P.local & 1, use = P.local >> 1;
        const int ti = kTile * t.i + rank, i = 128 * ti + r;
        const uint32_t tm = sh.tmem + acc * 256 + ((uint32_t)(32 * q) << 16);
        float4 dd[4];    // the chunk's values of A'
        if (PH == PH_S) {
            const int c = 64 * t.cb0 + 16 * turn, tj = kTile * t.j + (c >> 7);
            if (turn < 4 * t.nb && ti <= tj) {
                float* dt = gram_tile(M, ti, tj);
#pragma unroll
                for (int e = 0; e < 4; ++e) dd[e] = *tile_at(dt, r, (c & 127) + 4 * e);
            }
        }
        uint32_t xh[8];  // the chunk's operand values of X, chunks of eight in stored order, and the rest
        uint4 xr;
        if (PH == PH_U && turn < 4 * t.nb) {
            load_row16(M.xh[cur], i, 64 * t.cb0 + 16 * turn, M.cb, xh);
            xr = *rest_at(M, i, 64 * t.cb0 + 16 * turn);
        }
        if (!mbar_wait(&sh.tfull[acc], use & 1, &sh.abort, J.wait_ns, J.status, WAIT_EPI_TMEM_FULL)) return;
        tc_fence_after();
        for (int ch = turn; ch < 4 * t.nb; ch += kTurn) {
            uint32_t v[32];  // the first 16
            tmem_ld16(tm + 16 * ch, v);
            const int c = 64 * t.cb0 + 16 * ch;
            if (PH == PH_G) {
                tmem_ld_wait();
                if (t.slot >= 0) {
                    // 128 columns at a time, as phase R takes them
                    float* part = J.part + ((int64_t)t.slot * kTile + rank) * kTile * kTileF;
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *tile_at(part, r, c + e) = make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]),
                                                               __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                } else {
                    const int tj = kTile * t.j + (c >> 7);
                    if (ti <= tj) {
                        const int j = 128 * tj + (c & 127);
                        const float inv2 = 1.f / (M.tau * M.tau);
                        float o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(v[e]) * inv2 - (i == j + e && i < M.k ? sc.alpha : 0.f);
                        store_gram16(M, gram_tile(M, ti, tj), r, c & 127, i, j, ti != tj, o);
                    }
                }
            } else if (PH == PH_S) {
                const int tj = kTile * t.j + (c >> 7);
                const float bb = fmaf(2.f * J.c, sc.alpha, J.b);
                float4 d4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) d4[e] = dd[e];
                const int c2 = c + 16 * kTurn, tj2 = kTile * t.j + (c2 >> 7);
                if (ch + kTurn < 4 * t.nb && ti <= tj2) {
                    float* dt = gram_tile(M, ti, tj2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dd[e] = *tile_at(dt, r, (c2 & 127) + 4 * e);
                }
                tmem_ld_wait();
                if (ti <= tj) {
                    float o[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[4 * e] = fmaf(bb, d4[e].x, J.c * __uint_as_float(v[4 * e]));
                        o[4 * e + 1] = fmaf(bb, d4[e].y, J.c * __uint_as_float(v[4 * e + 1]));
                        o[4 * e + 2] = fmaf(bb, d4[e].z, J.c * __uint_as_float(v[4 * e + 2]));
                        o[4 * e + 3] = fmaf(bb, d4[e].w, J.c * __uint_as_float(v[4 * e + 3]));
                    }
                    const int j = 128 * tj + (c & 127);
                    store_row16(M.bp, i, j, M.rb, o);
                    if (ti != tj) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) M.bp[blocked(j + e, i, M.rb)] = __float2half_rn(o[e]);
                    }
                }
            } else {
                const int j = c;
                const float wx = J.a + sc.theta, wh = sc.beta - sc.theta;
                float h[16], y[16];
                const uint32_t rest[4] = {xr.x, xr.y, xr.z, xr.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t p = i & 1 ? xh[e + 4] : xh[e], q = i & 1 ? xh[e] : xh[e + 4];
                    unpack2_f16(p, h[2 * e], h[2 * e + 1]);
                    unpack2_f16(q, h[2 * e + 8], h[2 * e + 9]);
                }
                if (ch + kTurn < 4 * t.nb) {
                    load_row16(M.xh[cur], i, j + 16 * kTurn, M.cb, xh);
                    xr = *rest_at(M, i, j + 16 * kTurn);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = fmaf(wx, with_rest(h[e], rest[e >> 2], e & 3), wh * h[e]);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] += __uint_as_float(v[e]);
                if (step + 1 < J.steps) {
                    const uint4 p = pack8_f16(y), q = pack8_f16(y + 8);
                    store_row16(M.xh[cur ^ 1], i, j, M.cb, p, q);
                    const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) unpack2_f16(w[e], h[2 * e], h[2 * e + 1]);
                    *rest_at(M, i, j) = make_uint4(pack_rest4(y, h), pack_rest4(y + 4, h + 4), pack_rest4(y + 8, h + 8),
                                                   pack_rest4(y + 12, h + 12));
                } else if (i < M.k) {
                    write_result<16>(M, 0, i, j, y);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (PAIR)
                arrive_first(&sh.tempty[acc]);
            else
                mbar_arrive(&sh.tempty[acc]);
        }
    }
}

template <int PH, bool PAIR>
__device__ __forceinline__ void product_phase(const Job& J, int cur, int step, Shared& sh, uint8_t* ring, Pipe& P) {
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        produce<PH, PAIR>(J, cur, sh, ring, P);
    } else if (warp == 1) {
        if ((threadIdx.x & 31) == 0) issue<PH, PAIR>(J, sh, ring, P);
    } else {
        epilogue<PH, PAIR>(J, cur, step, sh, P);
    }
    __syncwarp();
}

// X in operand form, with its rest, from u, a 64 x 64 block of a matrix a block: a thread makes eight values of a row at a time,
// with its lanes along the stored rows.  Instructions and memory about equally: 2048 x 8192 in 23 us (67 MB in, 50 MB out).
__global__ void __launch_bounds__(256) ns_convert_kernel(const __grid_constant__ Job J) {
    __shared__ float red[8];
    constexpr int kUnits = kBlk / 8;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int mat = 0;
    while (mat + 1 < J.count && (int)blockIdx.x >= J.mat[mat + 1].c0) ++mat;
    const Mat& M = J.mat[mat];
    float s = block_sum(M.norm, M.chunks, red), pre, inv;
    const int which = which_sum(s, J.eps);
    if (which) s = block_sum(M.norm + which * kNormChunks, M.chunks, red);
    scale_of(which, s, J.eps, M.tau, pre, inv);
    const int e = blockIdx.x - M.c0, bi = e / M.cb, bj = e % M.cb;
    for (int t = threadIdx.x; t < kUnits; t += 256) {
        const int r = M.tall ? t & 63 : t >> 3, c = 8 * (M.tall ? t >> 6 : t & 7);
        const int i = 64 * bi + r, j = 64 * bj + c;
        float y[8];
        if (M.vec && j < M.n && i < M.k) {  // rows of a multiple of eight values
            const int64_t at = (int64_t)i * M.n + j;
            if (M.f32) {
                const float4* g = reinterpret_cast<const float4*>(static_cast<const float*>(M.g) + at);
                const float4 p = g[0], q = g[1];
                y[0] = p.x, y[1] = p.y, y[2] = p.z, y[3] = p.w, y[4] = q.x, y[5] = q.y, y[6] = q.z, y[7] = q.w;
                if (M.m) {
                    const float4* m = reinterpret_cast<const float4*>(M.m + at);
                    const float4 mp = m[0], mq = m[1];
                    const float f[8] = {mp.x, mp.y, mp.z, mp.w, mq.x, mq.y, mq.z, mq.w};
#pragma unroll
                    for (int x = 0; x < 8; ++x) y[x] = J.nesterov ? fmaf(J.mu, f[x], y[x]) : f[x];
                }
            } else {
                const uint4 p = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(M.g) + at);
                const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) y[2 * x] = __uint_as_float(w[x] << 16), y[2 * x + 1] = __uint_as_float(w[x] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                y[x] = i < M.k && j + x < M.n ? load_u(M, J, M.tall ? (int64_t)(j + x) * M.k + i : (int64_t)i * M.n + j + x) : 0.f;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) y[x] = y[x] * pre * inv;
        const uint4 p = pack8_f16(y);
        *reinterpret_cast<uint4*>(M.xh[0] + blocked(i, j, M.cb)) = p;
        float h[8];
        unpack2_f16(p.x, h[0], h[1]), unpack2_f16(p.y, h[2], h[3]);
        unpack2_f16(p.z, h[4], h[5]), unpack2_f16(p.w, h[6], h[7]);
        reinterpret_cast<uint2*>(rest_at(M, i, j))[(j >> 3) & 1] = make_uint2(pack_rest4(y, h), pack_rest4(y + 4, h + 4));
    }
}

// A' of the tiles whose long axis was cut: the sum of the parts, in their order, less alpha on the diagonal.  A warp takes four
// columns of 32 ROWS rows of a 128 x 128 tile at a time.
template <bool PAIR, int ROWS>
__device__ __forceinline__ void join_phase(const Job& J, int step) {
    constexpr int kTile = PAIR ? 2 : 1, kGroups = kTileF / 4 / (32 * ROWS), kWarps = kThreads / 32;
    constexpr int64_t kApart = (int64_t)kTile * kTile * kTileF;
    const int lane = threadIdx.x & 31, total = J.cuts * kTile * kTile * kGroups;
    for (int it = blockIdx.x * kWarps + (threadIdx.x >> 5); it < total; it += gridDim.x * kWarps) {
        const int in = it % kGroups, sub = it / kGroups % (kTile * kTile);
        const Cut& t = J.cut[it / (kTile * kTile * kGroups)];
        const Mat& M = J.mat[t.mat];
        const int ti = kTile * t.i + sub / kTile, tj = kTile * t.j + sub % kTile;
        if (ti > tj) continue;
        const int r = in * 32 * ROWS % 128 + lane, c = in * 32 * ROWS / 128 * 4;
        float* part = J.part + (int64_t)(2 * t.unit + 1) * kApart + sub * kTileF;
        float4 s[ROWS];
#pragma unroll
        for (int a = 0; a < ROWS; ++a) s[a] = *tile_at(part, r + 32 * a, c);
        part -= kApart;
#pragma unroll(8 / ROWS)
        for (int w = 1; w < t.parts; ++w) {
            part += 2 * kApart;
#pragma unroll
            for (int a = 0; a < ROWS; ++a) {
                const float4 x = *tile_at(part, r + 32 * a, c);
                s[a].x += x.x, s[a].y += x.y, s[a].z += x.z, s[a].w += x.w;
            }
        }
        const float inv2 = 1.f / (M.tau * M.tau), alpha = alpha_of(J.a, J.cap, M.k, step);
        float* d = gram_tile(M, ti, tj);
#pragma unroll
        for (int a = 0; a < ROWS; ++a) {
            const int i = 128 * ti + r + 32 * a, j = 128 * tj + c;
            float o[4] = {s[a].x * inv2, s[a].y * inv2, s[a].z * inv2, s[a].w * inv2};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i == j + e && i < M.k) o[e] -= alpha;
            *tile_at(d, r + 32 * a, c) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint2*>(M.ad + blocked(i, j, M.rb)) = make_uint2(pack_f16(o[0], o[1]), pack_f16(o[2], o[3]));
            if (ti != tj) {
#pragma unroll
                for (int e = 0; e < 4; ++e) M.ad[blocked(j + e, i, M.rb)] = __float2half_rn(o[e]);
            }
        }
    }
}

// What bounds it.  On pairs, 2048 x 8192: of a step's 96 us G takes 25 and U 48, at 0.33 and 0.38 us for each 256 x 256 x 64 of a
// pair where the tensor cores' measured burst rate allows 0.33; the rest is R 10, S 13 and four barriers of 2.5 each.  All five
// steps and the input passes: 541 us, 1.03 PFLOP/s.  (U's loads come to 113 bytes a nanosecond and SM, of 138 that L2 was measured
// to give.)  On single CTAs, small sizes: 300 x 2000 is 4.6 + 3.4 + 4.7 + 5.2 us a step, of which 2.5 each are the barrier and
// most of the rest the latency of loads, products and epilogue one after the other; S's and U's tiles are as narrow as fills the SMs (at 128 and 256 columns 116 us in place of 91).
// Waiting for a tile's parts in place of R and its barrier was slower (three of 515 x 1511, a step: 12.5 us for G and R against
// 12.1), as its reads are then a CTA's own and come late.
template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) ns_kernel(const __grid_constant__ Job J) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5;
    const bool first = !PAIR || cluster_rank() == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMostStages; ++s) {
            mbar_init(&sh.full[s], PAIR && first ? 2 : 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh.tfull[a], 1);
            mbar_init(&sh.tempty[a], (PAIR ? 2 : 1) * kEpiWarps);
        }
        mbar_init(&sh.drain, 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"(512) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            tmem_alloc(&sh.tmem, 512);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (PAIR)
        cluster_sync();  // the barriers of both CTAs are there
    else
        __syncthreads();
    tc_fence_after();

    Pipe P;
    uint32_t target = 0;
    bool ok = true;
    for (int step = 0; ok && step < J.steps; ++step) {
        const int cur = step & 1;
        product_phase<PH_G, PAIR>(J, cur, step, sh, ring, P);
        if (!(ok = grid_sync(J, target, sh))) break;
        if (J.cuts > 0) {
            // four rows to a lane where that leaves items for all warps
            if (J.cuts * (PAIR ? 128 : 32) >= (int)gridDim.x * kThreads / 32)
                join_phase<PAIR, 4>(J, step);
            else
                join_phase<PAIR, 1>(J, step);
            if (!(ok = grid_sync(J, target, sh))) break;
        }
        product_phase<PH_S, PAIR>(J, cur, step, sh, ring, P);
        if (!(ok = grid_sync(J, target, sh))) break;
        product_phase<PH_U, PAIR>(J, cur, step, sh, ring, P);
        if (step + 1 < J.steps) ok = grid_sync(J, target, sh);
    }
    // after a wait that gave up: copies and products in flight end before the CTA leaves
    if (*(volatile int*)&sh.abort) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < kMostStages; ++s)  // bits: the parity after a stage's last copy
                if (P.issued & (1u << s)) mbar_wait_timed(&sh.full[s], ((P.bits >> s) & 1) ^ 1, J.wait_ns);
        } else if (threadIdx.x == 32 && first) {
            if (PAIR)
                commit_pair(&sh.drain);
            else
                umma_commit(&sh.drain);
            mbar_wait_timed(&sh.drain, 0, J.wait_ns);
        }
    }
    tc_fence_before();
    if (PAIR)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512) : "memory");
        else
            tmem_dealloc(sh.tmem, 512);
    }
}

// A launch for matrices that a CTA or a cluster takes whole, of N kinds (arguments with room for 48 take their time: a lone call of
// 16 x 108 is 23 us with the host's part, with room for one 21.5).
template <int N>
struct SmallJob {
    Mat mat[N];
    int uniform;       // all matrices are like mat[0], `stride` values apart
    int64_t stride;
    int cluster;       // CTAs of a matrix
    int steps;
    float a, b, c, eps, mu, cap;
    int nesterov;
    int* status;
    uint64_t wait_ns;
};

// ---------------------------------------------------------------------------
// Matrices of at most K = 16 or 32 rows (the shorter side) that a CTA's shared memory holds twice: a CTA to a matrix, all of it
// in fp32 and without tensor cores, whose way in and out of tensor memory takes longer than these products.
//   A = X X^T: a group of lanes to a 4 x 4 tile on or above the diagonal, along the columns, then their sums
//   B = a I + b A + c A A: an entry to a thread
//   X = B X, into the other buffer: 4 x 4 entries to a thread (shared memory's bytes bound this: a column of eight took 1.8 times)
// One of 16 x 108 in 11 us (28.7 by the kernel below), of which about three are the loads and the norm; a step's bound is
// the latency of its three products, their sums over lanes and three block-wide barriers.

template <int K>
struct Tiny {
    static constexpr int kTiles = K / 4 * (K / 4 + 1) / 2, kLanes = K == 16 ? 32 : 16, kThreads = kTiles * kLanes;
    static constexpr int kLd = K + 4;                                  // a row of A and B in shared memory
    // Columns, at most.  A call here against the clusters below, which round to fp16: 16 x 108 12 : 29 us, 16 x 1024 42 : 39,
    // 16 x 1408 53 : 38, 16 x 1500 57 : 41, 32 x 108 20 : 29, 32 x 432 45 : 37, 32 x 512 51 : 37, 32 x 768 71 : 37.  So the last third
    // of these columns costs up to 15 us for results in fp32.
    static constexpr int kCols = K == 16 ? 1408 : 512;
    static constexpr size_t smem(int n) { return sizeof(float) * (2 * (size_t)K * ((n + 3) / 4 * 4 + 4) + 2 * K * kLd + 2 * 32); }
};

template <int K, int N>
__global__ void __launch_bounds__(Tiny<K>::kThreads) ns_tiny_kernel(const __grid_constant__ SmallJob<N> J) {
    using T = Tiny<K>;
    constexpr int kAhead = 8;  // loads of a thread in flight
    extern __shared__ __align__(16) float tiny_smem[];
    const int id = blockIdx.x, t = threadIdx.x;
    const Mat& M = J.mat[J.uniform ? 0 : id];
    const int64_t off = J.uniform ? id * J.stride : 0;
    const int k = M.k, n = M.n, n4 = (n + 3) / 4, ld = 4 * n4 + 4, count = k * n;
    float* x0 = tiny_smem;
    float* x1 = x0 + K * ld;
    float* A = x1 + K * ld;
    float* B = A + K * T::kLd;
    float* red = B + K * T::kLd;
    // of the stored element e; the quotient by d is exact while e d < 2^32
    const uint32_t d = M.tall ? k : n, part = 0xFFFFFFFFu / d + 1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // for the rest of a list
    auto place = [&](uint32_t e) {
        const uint32_t q = part ? __umulhi(e, part) : e, r = e - q * d;
        return M.tall ? r * ld + q : q * ld + r;
    };

    for (int e = t; e < K * ld; e += T::kThreads) x0[e] = 0.f;
    __syncthreads();
    float s = 0.f;
    for (int e0 = t; e0 < count; e0 += kAhead * T::kThreads) {
        float u[kAhead], m[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int e = e0 + a * T::kThreads;
            u[a] = m[a] = 0.f;
            if (e >= count) continue;
            u[a] = M.f32 ? static_cast<const float*>(M.g)[off + e] : bf16_bits_to_float(static_cast<const uint16_t*>(M.g)[off + e]);
            if (M.m) m[a] = M.m[off + e];
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int e = e0 + a * T::kThreads;
            if (e >= count) continue;
            if (M.m) {
                m[a] = fmaf(J.mu, m[a], u[a]);
                M.m[off + e] = m[a];
                u[a] = J.nesterov ? fmaf(J.mu, m[a], u[a]) : m[a];
            }
            s = fmaf(u[a], u[a], s);
            x0[place(e)] = u[a];
        }
    }
    auto total = [&](float v, float* to) {
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
        if ((t & 31) == 0) to[t >> 5] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < T::kThreads / 32; ++w) v += to[w];
        return v;
    };
    s = total(s, red);
    const int which = which_sum(s, J.eps);
    if (which) {
        s = 0.f;
        for (int e = t; e < K * ld; e += T::kThreads) {
            const float u = x0[e] * (which == 1 ? kDown : kUp);
            s = fmaf(u, u, s);
        }
        s = total(s, red + 32);
    }
    float pre, inv;
    scale_of(which, s, J.eps, 1.f, pre, inv);
    for (int e = t; e < K * ld; e += T::kThreads) x0[e] = x0[e] * pre * inv;
    __syncthreads();

    int ti, tj;  // the tile of the thread's group
    upper_tile(t / T::kLanes, K / 4, ti, tj);
    const int in = t % T::kLanes;
    for (int step = 0; step < J.steps; ++step) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        for (int c = in; c < n4; c += T::kLanes) {
            float4 p[4], q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[e] = *reinterpret_cast<const float4*>(x0 + (4 * ti + e) * ld + 4 * c);
                q[e] = *reinterpret_cast<const float4*>(x0 + (4 * tj + e) * ld + 4 * c);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float4 a = p[e >> 2], b = q[e & 3];
                v[e] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, v[e]))));
            }
        }
        // each exchange halves the entries that a lane sums on
#pragma unroll
        for (int o = 8; o; o >>= 1) {
            const bool up = in & o;
#pragma unroll
            for (int e = 0; e < o; ++e) {
                const float give = up ? v[e] : v[e + o], keep = up ? v[e + o] : v[e];
                v[e] = keep + __shfl_xor_sync(~0u, give, o);
            }
        }
        if (T::kLanes == 32) v[0] += __shfl_xor_sync(~0u, v[0], 16);
        if (in < 16) {
            const int i = 4 * ti + (in >> 2), j = 4 * tj + (in & 3);
            A[i * T::kLd + j] = v[0];
            A[j * T::kLd + i] = v[0];
        }
        __syncthreads();
        for (int e = t; e < K * K; e += T::kThreads) {
            const int i = e / K, j = e % K;
            float d = 0.f;
#pragma unroll
            for (int l = 0; l < K; l += 4) {
                const float4 a = *reinterpret_cast<const float4*>(A + i * T::kLd + l);
                const float4 b = *reinterpret_cast<const float4*>(A + j * T::kLd + l);
                d = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, d))));
            }
            B[i * T::kLd + j] = fmaf(J.b, A[i * T::kLd + j], fmaf(J.c, d, i == j ? J.a : 0.f));
        }
        __syncthreads();
        for (int e = t, c = t, i = 0; e < n4 * (K / 4); e += T::kThreads, c += T::kThreads) {
            while (c >= n4) c -= n4, i += 4;
            float4 y[4] = {};
#pragma unroll
            for (int l = 0; l < K; l += 4) {
                float4 x[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = *reinterpret_cast<const float4*>(x0 + (l + r) * ld + 4 * c);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 b = *reinterpret_cast<const float4*>(B + (i + r) * T::kLd + l);
                    y[r].x = fmaf(b.x, x[0].x, fmaf(b.y, x[1].x, fmaf(b.z, x[2].x, fmaf(b.w, x[3].x, y[r].x))));
                    y[r].y = fmaf(b.x, x[0].y, fmaf(b.y, x[1].y, fmaf(b.z, x[2].y, fmaf(b.w, x[3].y, y[r].y))));
                    y[r].z = fmaf(b.x, x[0].z, fmaf(b.y, x[1].z, fmaf(b.z, x[2].z, fmaf(b.w, x[3].z, y[r].z))));
                    y[r].w = fmaf(b.x, x[0].w, fmaf(b.y, x[1].w, fmaf(b.z, x[2].w, fmaf(b.w, x[3].w, y[r].w))));
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) *reinterpret_cast<float4*>(x1 + (i + r) * ld + 4 * c) = y[r];
        }
        __syncthreads();
        float* x = x0;
        x0 = x1;
        x1 = x;
    }
    for (int e0 = t; e0 < count; e0 += kAhead * T::kThreads) {
        float w[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int e = e0 + a * T::kThreads;
            w[a] = M.w && e < count ? M.w[off + e] : 0.f;
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int e = e0 + a * T::kThreads;
            if (e >= count) continue;
            float y = x0[place(e)];
            if (M.w) M.w[off + e] = y = M.keep * w[a] - M.step * y;
            if (M.o) M.o[off + e] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        }
    }
}

// ---------------------------------------------------------------------------
// Matrices of at most 128 rows (the shorter side): a cluster of CTAs to a matrix runs all of it without leaving the chip, each
// CTA on a slice of the columns.  X's slice is an operand in shared memory and, in fp32, an accumulator in tensor memory, onto
// which U's product is added in place.  The Gram matrix's parts are exchanged through the CTAs' shared memory: each CTA sums
// and rounds a slice of its columns for all, and A' A' and B' are then computed by every CTA for itself.
// Latency bounds it: a call of 64 x 432 takes 45 us and of 128 x 128 43, some 8 a step, one after the other three products with
// their ways in and out of tensor memory and, in clusters, two exchanges.

constexpr int kSmallThreads = 256;
constexpr int kSmallRows = 128, kSmallCols = 384;  // of a CTA: 128 tensor memory columns are left to the Gram matrix
constexpr int kMaxCluster = 16;
constexpr uint32_t kMaxShared = 1024 + (2 * kSmallCols / 64 + 8) * kBlkBytes + 4 * kTileF;
constexpr uint32_t kGram = 384;                    // its tensor memory column

struct SmallShared {
    uint64_t bar;
    uint32_t tmem;
    int abort;
    float red[24];
    float4 sums[kMaxCluster];  // of the CTAs: the three sums of u^2
};

// Byte offset of element (r, c) of a 128-row operand in shared memory: 64 x 64 blocks, a column's two blocks in turn.
__device__ __forceinline__ uint32_t small_at(int r, int c) {
    return (uint32_t)(((c >> 6) * 2 + (r >> 6)) * (int)kBlkBytes + (r & 63) * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4) + (c & 7) * 2);
}

// The three sums of all threads, to slot `rank` of every CTA of the cluster; visible after the next cluster_sync.
__device__ __forceinline__ void share_sums(SmallShared& sh, float a, float b, float c, int rank, int cluster) {
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(~0u, a, o);
        b += __shfl_xor_sync(~0u, b, o);
        c += __shfl_xor_sync(~0u, c, o);
    }
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sh.red[warp] = a, sh.red[8 + warp] = b, sh.red[16 + warp] = c;
    __syncthreads();
    if ((int)threadIdx.x < cluster) {
        a = b = c = 0.f;
        for (int i = 0; i < 8; ++i) a += sh.red[i], b += sh.red[8 + i], c += sh.red[16 + i];
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(remote(&sh.sums[rank], threadIdx.x)), "f"(a), "f"(b),
                     "f"(c), "f"(0.f)
                     : "memory");
    }
}
__device__ __forceinline__ float3 total_sums(const SmallShared& sh, int cluster) {
    float3 t = make_float3(0.f, 0.f, 0.f);
    for (int i = 0; i < cluster; ++i) {
        t.x += sh.sums[i].x;
        t.y += sh.sums[i].y;
        t.z += sh.sums[i].z;
    }
    return t;
}

template <int N>
__global__ void __launch_bounds__(kSmallThreads, 1) ns_small_kernel(const __grid_constant__ SmallJob<N> J) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ SmallShared sh;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int id = blockIdx.x / J.cluster, rank = (int)cluster_rank(), Q = J.cluster;
    const Mat& M = J.mat[J.uniform ? 0 : id];
    const int64_t off = J.uniform ? id * J.stride : 0;
    const int kr = (M.k + 31) / 32 * 32;                                     // rows that are worked on
    const int per = (M.cb + Q - 1) / Q, b0 = min(rank * per, M.cb), nb = min(per, M.cb - b0);  // 64-column blocks of the CTA
    const int j0 = 64 * b0;
    uint8_t* xh = smem;                              // 128 rows of X's operand
    uint8_t* ad = smem + per * 2 * kBlkBytes;        // A', then B': 128 x 128
    uint8_t* al = ad + 4 * kBlkBytes;                // what rounding left of A'
    float4* recv = reinterpret_cast<float4*>(al + 4 * kBlkBytes);  // the other CTAs' parts of this one's slice of the Gram matrix
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, half = warp >> 2;
    const int i = 32 * q + lane;
    const bool rows = 32 * q < kr;                   // the warp's rows are worked on
    uint32_t phase = 0;

    if (threadIdx.x == 0) {
        mbar_init(&sh.bar, 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    // rows beyond those worked on stay zero
    for (int t = threadIdx.x; t < nb * 2 * (int)kBlkBytes / 16; t += kSmallThreads) reinterpret_cast<uint4*>(xh)[t] = make_uint4(0, 0, 0, 0);
    for (int t = threadIdx.x; t < 8 * (int)kBlkBytes / 16; t += kSmallThreads) reinterpret_cast<uint4*>(ad)[t] = make_uint4(0, 0, 0, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh.tmem + ((uint32_t)(32 * q) << 16);
    auto wait = [&]() {
        mbar_wait(&sh.bar, phase & 1, &sh.abort, J.wait_ns, J.status, WAIT_MMA_FULL);
        ++phase;
        tc_fence_after();
    };

    // u into tensor memory, with the momentum step, and the sums of its squares
    float s = 0.f, s2 = 0.f, s3 = 0.f;
    if (rows)
        for (int ch = half; ch < 2 * nb; ch += 2) {
            uint32_t v[32];
            const int j = j0 + 32 * ch;
            const int64_t base = off + (M.tall ? (int64_t)j * M.k + i : (int64_t)i * M.n + j), st = M.tall ? M.k : 1;
            float u[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const bool in = i < M.k && j + e < M.n;
                u[e] = !in ? 0.f
                           : M.f32 ? static_cast<const float*>(M.g)[base + e * st]
                                   : bf16_bits_to_float(static_cast<const uint16_t*>(M.g)[base + e * st]);
            }
            if (M.m) {
                float m[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) m[e] = i < M.k && j + e < M.n ? M.m[base + e * st] : 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    m[e] = fmaf(J.mu, m[e], u[e]);
                    if (i < M.k && j + e < M.n) M.m[base + e * st] = m[e];
                    u[e] = J.nesterov ? fmaf(J.mu, m[e], u[e]) : m[e];
                }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                add_squares(u[e], s, s2, s3);
                v[e] = __float_as_uint(u[e]);
            }
            tmem_st32(tm + 32 * ch, v);
        }
    tmem_st_wait();
    cluster_sync();  // every CTA of the cluster has begun
    share_sums(sh, s, s2, s3, rank, Q);
    cluster_sync();
    const float3 uu = total_sums(sh, Q);
    const int which = which_sum(uu.x, J.eps);
    float pre, inv;
    scale_of(which, which == 1 ? uu.y : which == 2 ? uu.z : uu.x, J.eps, M.tau, pre, inv);
    if (rows)
        for (int ch = half; ch < 2 * nb; ch += 2) {
            uint32_t v[32];
            tmem_ld32(tm + 32 * ch, v);
            tmem_ld_wait();
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                y[e] = __uint_as_float(v[e]) * pre * inv;
                v[e] = __float_as_uint(y[e]);
            }
            tmem_st32(tm + 32 * ch, v);
#pragma unroll
            for (int e = 0; e < 32; e += 8) *reinterpret_cast<uint4*>(xh + small_at(i, 32 * ch + e)) = pack8_f16(&y[e]);
        }
    tmem_st_wait();
    const float inv2 = 1.f / (M.tau * M.tau);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();

    const int w = kSmallRows / Q;  // columns of the Gram matrix that a CTA sums
    for (int step = 0; step < J.steps; ++step) {
        if (threadIdx.x == 0) {
            tc_fence_after();
            const uint32_t xs = smem_u32(xh), id16 = idesc_f16(128, kr, 0);
            for (int kk = 0; kk < 4 * nb; ++kk) {
                const uint64_t d = sdesc(xs + (kk >> 2) * 2 * kBlkBytes + (kk & 3) * 32, 16, 1024, SWZ_128B);
                umma_bf16(sh.tmem + kGram, d, d, id16, kk > 0);
            }
            umma_commit(&sh.bar);
        }
        __syncwarp();
        wait();
        const float alpha = alpha_of(J.a, J.cap, M.k, step);
        if (Q == 1) {
            if (rows)
                for (int ch = half; ch < kr / 32; ch += 2) {
                    uint32_t v[32];
                    tmem_ld32(tm + kGram + 32 * ch, v);
                    tmem_ld_wait();
                    float h[32], l[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float d = __uint_as_float(v[e]) * inv2 - (i == 32 * ch + e && i < M.k ? alpha : 0.f);
                        h[e] = __half2float(__float2half_rn(d));
                        l[e] = d - h[e];
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        *reinterpret_cast<uint4*>(ad + small_at(i, 32 * ch + e)) = pack8_f16(&h[e]);
                        *reinterpret_cast<uint4*>(al + small_at(i, 32 * ch + e)) = pack8_f16(&l[e]);
                    }
                }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncthreads();
        } else {
            if (rows && nb > 0)
                for (int ch = half; ch < kr / 32; ch += 2) {
                    uint32_t v[32];
                    tmem_ld32(tm + kGram + 32 * ch, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const int c = 32 * ch + e;
                        const uint32_t at = remote(recv + (rank * (w / 4) + (c % w) / 4) * 128 + i, c / w);
                        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[e]), "r"(v[e + 1]), "r"(v[e + 2]),
                                     "r"(v[e + 3])
                                     : "memory");
                    }
                }
            tc_fence_before();
            cluster_sync();
            // the slice of all CTAs that have columns, in turn
            const int have = (M.cb + per - 1) / per, r = threadIdx.x & 127;
            if (r < kr && rank * w < kr)
                for (int c4 = threadIdx.x >> 7; c4 < w / 4; c4 += 2) {
                    float4 t = recv[c4 * 128 + r];
                    for (int o = 1; o < have; ++o) {
                        const float4 x = recv[(o * (w / 4) + c4) * 128 + r];
                        t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
                    }
                    const int j = rank * w + 4 * c4;
                    float d[4] = {t.x * inv2, t.y * inv2, t.z * inv2, t.w * inv2}, h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (r == j + e && r < M.k) d[e] -= alpha;
                        h[e] = __half2float(__float2half_rn(d[e]));
                    }
                    const uint32_t h0 = pack_f16(h[0], h[1]), h1 = pack_f16(h[2], h[3]);
                    const uint32_t l0 = pack_f16(d[0] - h[0], d[1] - h[1]), l1 = pack_f16(d[2] - h[2], d[3] - h[3]);
                    const uint32_t at = small_at(r, j);
                    for (int o = 0; o < have; ++o) {
                        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(remote(ad + at, o)), "r"(h0), "r"(h1) : "memory");
                        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(remote(al + at, o)), "r"(l0), "r"(l1) : "memory");
                    }
                }
            fence_async();
            cluster_sync();
        }
        const float beta = alpha * fmaf(J.c, alpha, J.b), theta = step + 2 >= J.steps ? beta : 0.f;
        const float wx = J.a + theta, wh = beta - theta, bb = fmaf(2.f * J.c, alpha, J.b);
        if (threadIdx.x == 0) {
            tc_fence_after();
            fence_proxy_async_smem();
            const uint32_t as = smem_u32(ad), id16 = idesc_f16(128, kr, 0);
            for (int kk = 0; kk < kr / 16; ++kk) {
                const uint64_t d = sdesc(as + (kk >> 2) * 2 * kBlkBytes + (kk & 3) * 32, 16, 1024, SWZ_128B);
                umma_bf16(sh.tmem + kGram, d, d, id16, kk > 0);
            }
            umma_commit(&sh.bar);
        }
        __syncwarp();
        // meanwhile what X itself contributes to its successor
        if (rows)
            for (int ch = half; ch < 2 * nb; ch += 2) {
                uint32_t v[32];
                tmem_ld32(tm + 32 * ch, v);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float y = __uint_as_float(v[e]);
                    v[e] = __float_as_uint(fmaf(wx, y, wh * __half2float(__float2half_rn(y))));
                }
                tmem_st32(tm + 32 * ch, v);
            }
        tmem_st_wait();
        wait();
        if (rows)
            for (int ch = half; ch < kr / 32; ch += 2) {
                uint32_t v[32];
                tmem_ld32(tm + kGram + 32 * ch, v);
                uint4 h4[4], l4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h4[e] = *reinterpret_cast<const uint4*>(ad + small_at(i, 32 * ch + 8 * e));
                    l4[e] = *reinterpret_cast<const uint4*>(al + small_at(i, 32 * ch + 8 * e));
                }
                tmem_ld_wait();
                float o[32];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t hw[4] = {h4[e].x, h4[e].y, h4[e].z, h4[e].w}, lw[4] = {l4[e].x, l4[e].y, l4[e].z, l4[e].w};
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&hw[p]));
                        const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&lw[p]));
                        const int f = 8 * e + 2 * p;
                        o[f] = fmaf(bb, fh.x + fl.x, J.c * __uint_as_float(v[f]));
                        o[f + 1] = fmaf(bb, fh.y + fl.y, J.c * __uint_as_float(v[f + 1]));
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) *reinterpret_cast<uint4*>(ad + small_at(i, 32 * ch + e)) = pack8_f16(&o[e]);
            }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (threadIdx.x == 0) {
            tc_fence_after();
            const uint32_t as = smem_u32(ad), xs = smem_u32(xh);
            for (int kk = 0; kk < kr / 16; ++kk) {
                const uint64_t da = sdesc(as + (kk >> 2) * 2 * kBlkBytes + (kk & 3) * 32, 16, 1024, SWZ_128B);
                for (int c = 0; c < nb; c += 4)
                    umma_bf16(sh.tmem + 64 * c, da,
                              sdesc(xs + c * 2 * kBlkBytes + (kk >> 2) * kBlkBytes + (kk & 3) * 2048, 2 * kBlkBytes, 1024, SWZ_128B),
                              idesc_f16(128, 64 * min(4, nb - c), 1), 1u);
            }
            umma_commit(&sh.bar);
        }
        __syncwarp();
        wait();
        const bool last = step + 1 == J.steps;
        if (rows)
            for (int ch = half; ch < 2 * nb; ch += 2) {
                uint32_t v[32];
                tmem_ld32(tm + 32 * ch, v);
                tmem_ld_wait();
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(v[e]);
                if (!last) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) *reinterpret_cast<uint4*>(xh + small_at(i, 32 * ch + e)) = pack8_f16(&y[e]);
                } else if (i < M.k) {
                    write_result<32>(M, off, i, j0 + 32 * ch, y);
                }
            }
        if (!last) {
            // (a cluster's CTAs write each other's A' only after the next exchange's first barrier)
            fence_proxy_async_smem();
            tc_fence_before();
            __syncthreads();
        }
    }
    if (sh.abort && threadIdx.x == 0) {  // products in flight end before the CTA leaves
        umma_commit(&sh.bar);
        mbar_wait_timed(&sh.bar, phase & 1, J.wait_ns);
    }
    if (threadIdx.x == 0) after_previous();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, 512);
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool shape_ok(int64_t rows, int64_t cols) { return rows > 0 && cols > 0; }
bool shape_supported(int64_t rows, int64_t cols) { return rows <= 65536 && cols <= 65536; }

struct Poly {
    int steps;
    float a, b, c, eps;
};
bool poly_ok(const Poly& p) {
    return p.steps >= 1 && std::isfinite(p.a) && std::isfinite(p.b) && std::isfinite(p.c) && p.eps >= 0.f && std::isfinite(p.eps);
}

// The squared singular value that the polynomial leaves in place, the smallest root of a + b t + c t^2 = 1 in (0, 2]; 0 (alpha is
// not used) where there is none.
float cap_of(const Poly& p) {
    const double a = p.a - 1.0, b = p.b, c = p.c;
    double best = 0.0;
    auto take = [&](double t) {
        if (t > 0.0 && t <= 2.0 && (best == 0.0 || t < best)) best = t;
    };
    if (c == 0.0) {
        if (b != 0.0) take(-a / b);
    } else if (b * b >= 4.0 * a * c) {
        const double r = std::sqrt(b * b - 4.0 * a * c);
        take((-b - r) / (2.0 * c));
        take((-b + r) / (2.0 * c));
    }
    return (float)best;
}

// Pairs of CTAs take a launch whose update products have this many tiles of 256 x 256, counted by their blocks of 64 contracted
// values, or more: a pair loads less a product and waits longer at each step of its ring.  A whole call, single CTAs against pairs:
// 2048 x 2048 (2048 blocks) 244 : 241 us, 1024 x 8192 (2048) 264 : 274, the seven convolutions' filters (2400) 361 : 376,
// 2048 x 3000 (3072) 307 : 303, 1500 x 8192 (4608) 410 : 382, 2048 x 8192 (8192) 589 : 545.
constexpr int64_t kPairWork = 2700;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Sizes, and the split of the long axis, of matrices that run in one launch; returns whether on pairs of CTAs.
bool plan_sizes(Mat* mats, int count) {
    int64_t work = 0;
    for (int i = 0; i < count; ++i) {
        Mat& M = mats[i];
        M.tall = M.rows > M.cols;
        M.k = (int)std::min(M.rows, M.cols), M.n = (int)std::max(M.rows, M.cols);
        M.vec = !M.tall && M.n % 8 == 0;
        M.wide = !M.tall && M.n % 16 == 0 && (reinterpret_cast<uintptr_t>(M.w) | reinterpret_cast<uintptr_t>(M.o)) % 32 == 0;
        M.aligned = reinterpret_cast<uintptr_t>(M.g) % 16 == 0;
        M.nx = (M.n + 63) / 64;
        work += (int64_t)((M.k + 255) / 256) * ((M.nx + 3) / 4) * ((M.k + 63) / 64);
    }
    const bool pair = work >= kPairWork;
    const int tile = pair ? 2 : 1;
    for (int i = 0; i < count; ++i) {
        Mat& M = mats[i];
        M.cb = pair ? (M.nx + 3) / 4 * 4 : M.nx;
        M.gt = (M.k + 128 * tile - 1) / (128 * tile), M.mt = tile * M.gt, M.rb = 2 * M.mt;
        const int64_t total = M.rows * M.cols;
        M.chunk = std::max<int64_t>(4096, ((total + kNormChunks - 1) / kNormChunks + 3) / 4 * 4);
        M.chunks = (int)((total + M.chunk - 1) / M.chunk);
        // entries of X are 1 / sqrt(k n) at first and at most about 1.2 / sqrt(n) in the mean later: a quarter of the former's inverse
        M.tau = std::exp2(std::floor(std::log2(std::max(4.0, std::sqrt((double)M.k * M.n)) / 4.0)));
    }
    return pair;
}

// How phase G's tiles are dealt out: whole or in halves of their columns, in turn, or (returns a unit's share) cut into even shares
// of all blocks.  In loads of an operand block, of which an SM takes one in 0.058 us: a block of the contracted axis takes four, in
// a half three, and a cut 64 more, phase R and its barrier.  (A step's G and R, cut against halves: three of 515 x 1511 12.1 : 11.1
// us, 1024 x 1024 11.5 : 8.5; cut, 300 x 2000 takes 8.4 and 512 x 2048 9.3.)
int gram_share(const Mat* mats, int count, bool pair, int* half) {
    const int units = kPlanSms / (pair ? 2 : 1);
    std::vector<int64_t> load((size_t)units);
    int64_t blocks = 0, best = INT64_MAX;
    for (int h = 0; h < 2; ++h) {
        std::fill(load.begin(), load.end(), 0);
        size_t u = 0;
        for (int i = 0; i < count; ++i) {
            const int64_t tiles = (int64_t)mats[i].gt * (mats[i].gt + 1) / 2;
            if (h == 0) blocks += tiles * mats[i].nx;
            for (int64_t t = 0; t < tiles << h; ++t) {
                load[u] += mats[i].nx;
                if (++u == load.size()) u = 0;
            }
        }
        const int64_t most = (4 - h) * *std::max_element(load.begin(), load.end());
        if (most < best) best = most, *half = h;
    }
    const int64_t share = std::max<int64_t>(4, (blocks + units - 1) / units);
    return best <= 4 * share + 64 ? 0 : (int)share;
}

// 64-column blocks of a tile of phase U on single CTAs, which keep the busiest CTA least: a tile takes as long as its blocks'
// loads (2 + width for each contracted block) and an epilogue that was measured to be worth ten loads a block of width.
int update_width(const Mat* mats, int count) {
    int64_t best = INT64_MAX;
    int width = 4;
    std::vector<int64_t> load((size_t)kPlanSms);
    for (int w = 4; w >= 1; --w) {
        std::fill(load.begin(), load.end(), 0);
        size_t u = 0;
        for (int i = 0; i < count; ++i)
            for (int64_t t = (int64_t)mats[i].gt * ((mats[i].nx + w - 1) / w); t > 0; --t) {
                load[u] += (int64_t)((mats[i].k + 63) / 64) * (2 + w) + 10 * w + 8;
                if (++u == load.size()) u = 0;
            }
        const int64_t most = *std::max_element(load.begin(), load.end());
        if (most < best) best = most, width = w;
    }
    return width;
}

// The tiles that the ends of shares lie in.
void list_cuts(Job& J) {
    int last = -1, mat = 0;
    for (int b = J.share; b < J.blocks; b += J.share) {
        while (mat + 1 < J.count && b >= J.mat[mat + 1].b0) ++mat;
        const Mat& M = J.mat[mat];
        int e = (b - M.b0) / M.nx;
        const int first = M.b0 + e * M.nx;
        if (b == first || first == last) continue;  // between tiles, or a tile that is listed
        last = first;
        Cut& t = J.cut[J.cuts++];
        t.mat = (int16_t)mat;
        t.unit = (uint8_t)(first / J.share);
        t.parts = (uint8_t)((first + M.nx - 1) / J.share - t.unit + 1);
        int i = 0;
        for (; e >= M.gt - i; ++i) e -= M.gt - i;
        t.i = (int16_t)i, t.j = (int16_t)(i + e);
    }
}

// Places the matrices' buffers and the parts after the first 256 bytes of `base` (which may be NULL, to count) and returns the
// size that this takes of a workspace that starts at any 16 bytes: the operands are accessed 32 bytes at a time, and begin at
// multiples of 256.
size_t place(Mat* mats, int count, bool pair, char* base, float** part) {
    size_t at = 256;
    base += (256 - reinterpret_cast<uintptr_t>(base) % 256) % 256;
    auto take = [&](size_t bytes) {
        char* p = base + at;
        at += up256(bytes);
        return p;
    };
    for (int i = 0; i < count; ++i) {
        Mat& M = mats[i];
        const size_t xb = (size_t)M.rb * M.cb * kBlkBytes, ab = (size_t)M.rb * M.rb * kBlkBytes;
        for (int p = 0; p < 2; ++p) M.xh[p] = reinterpret_cast<__half*>(take(xb));
        M.x = reinterpret_cast<uint8_t*>(take(xb / 2));
        M.ad = reinterpret_cast<__half*>(take(ab));
        M.bp = reinterpret_cast<__half*>(take(ab));
        M.d = reinterpret_cast<float*>(take((size_t)M.mt * (M.mt + 1) / 2 * kTileF * sizeof(float)));
        M.norm = reinterpret_cast<float*>(take(3 * kNormChunks * sizeof(float)));
    }
    int half;
    *part = reinterpret_cast<float*>(take(gram_share(mats, count, pair, &half) ? 2 * kPlanSms * (pair ? 2 : 1) * kTileF * sizeof(float) : 0));
    return at + 256 - 16;
}

// CTAs of a matrix in ns_small_kernel, 0 where it does not take the matrix: as many as leave a CTA about two blocks of 64 columns,
// or four where there are more than 64 rows (the exchange then weighs as much), and one where it holds them all but for that.
// A call, two blocks against four: 64 x 432 45 : 53 us, 64 x 2000 56 : 61, 128 x 432 71 : 72, 128 x 1024 85 : 88, 128 x 1536
// 123 : 92.  Long matrices go to ns_kernel, here against there: 64 x 2000 56 : 88, 64 x 4096 67 : 94, 128 x 432 72 : 76,
// 128 x 1024 88 : 86, 128 x 1536 92 : 96, 128 x 1728 94 : 91, 128 x 3456 132 : 92.
int cluster_of(const Mat& M) {
    const int64_t k = std::min(M.rows, M.cols), n = std::max(M.rows, M.cols), cb = (n + 63) / 64, each = k > 64 ? 4 : 2;
    if (k > kSmallRows || n > (k > 64 ? 1536 : 4096)) return 0;
    int q = 1;
    if (cb > (k > 64 ? kSmallCols / 64 : each))
        while (q < kMaxCluster && each * q < cb) q *= 2;
    return q;
}

// Matrices that all fit ns_small_kernel go there: the CTAs of a cluster, else 0.  (Beside larger ones they cost little.)
int cluster_of(const std::vector<Mat>& mats) {
    int most = 0;
    for (const Mat& M : mats) {
        const int q = cluster_of(M);
        if (q == 0) return 0;
        most = std::max(most, q);
    }
    return most;
}

// The K of ns_tiny_kernel that takes all of the matrices, or 0.
int tiny_of(const std::vector<Mat>& mats) {
    int64_t k = 0, n = 0;
    for (const Mat& M : mats) k = std::max(k, std::min(M.rows, M.cols)), n = std::max(n, std::max(M.rows, M.cols));
    return k <= 16 && n <= Tiny<16>::kCols ? 16 : k <= 32 && n <= Tiny<32>::kCols ? 32 : 0;
}

// Takes the matrices of at most 16 rows and 512 columns out of a list that has larger ones: ns_tiny_kernel takes them in fp32.  With
// fp16 operands what a few values' rounding does depends on the matrix, up to 1e-2 of the result for 3 x 3 and 5e-3 for 4 x 8, where
// many values' is 1e-3.  Up to 25 us, of which most lie under the other matrices' input pass.
std::vector<Mat> take_few(std::vector<Mat>& mats) {
    std::vector<Mat> few;
    if (tiny_of(mats)) return few;
    const auto rest = std::stable_partition(mats.begin(), mats.end(), [](const Mat& M) {
        return std::min(M.rows, M.cols) > 16 || std::max(M.rows, M.cols) > 512;
    });
    few.assign(rest, mats.end());
    mats.erase(rest, mats.end());
    return few;
}

size_t workspace_of(std::vector<Mat>& mats) {
    if (cluster_of(mats)) return 256;
    size_t most = 0;
    for (size_t b = 0; b < mats.size(); b += kMaxMats) {
        const int count = (int)std::min<size_t>(kMaxMats, mats.size() - b);
        const bool pair = plan_sizes(&mats[b], count);
        float* part;
        most = std::max(most, place(&mats[b], count, pair, nullptr, &part));
    }
    return most;
}

// The runtime's error is taken with its report: the next call is not to find it.
cf_status cuda_error() {
    cudaGetLastError();
    return CF_ERR_CUDA;
}

// A launch that may begin before the one before it in the stream has ended.
cudaLaunchAttribute overlap() {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    return at;
}

// beside: the first launch may run beside the one before it.
template <int N>
cf_status run_small(const LaunchCtx& ctx, const Poly& p, float mu, int nesterov, std::vector<Mat>& mats, int cluster, bool uniform,
                    bool beside) {
    const int tiny = tiny_of(mats);
    const auto kernel = tiny == 16 ? ns_tiny_kernel<16, N> : tiny == 32 ? ns_tiny_kernel<32, N> : ns_small_kernel<N>;
    if (tiny) cluster = 1;
    const size_t most = tiny == 16 ? Tiny<16>::smem(Tiny<16>::kCols) : tiny == 32 ? Tiny<32>::smem(Tiny<32>::kCols) : kMaxShared;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess ||
        (cluster > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess))
        return cuda_error();
    const size_t each = uniform ? mats.size() : N;
    for (size_t b = 0; b < mats.size(); b += each) {
        SmallJob<N> J{};
        const int count = (int)std::min(each, mats.size() - b);
        int per = 1, longest = 1;
        plan_sizes(&mats[b], uniform ? 1 : count);
        for (int i = 0; i < (uniform ? 1 : count); ++i) {
            J.mat[i] = mats[b + i];
            per = std::max(per, (mats[b + i].cb + cluster - 1) / cluster);
            longest = std::max(longest, mats[b + i].n);
        }
        J.uniform = uniform, J.stride = mats[0].rows * mats[0].cols;
        J.cluster = cluster;
        J.steps = p.steps, J.a = p.a, J.b = p.b, J.c = p.c, J.eps = p.eps, J.cap = cap_of(p), J.mu = mu, J.nesterov = nesterov;
        J.status = ctx.status;
        J.wait_ns = ctx.wait_ns;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(count * cluster));
        cfg.blockDim = dim3(tiny == 16 ? Tiny<16>::kThreads : tiny == 32 ? Tiny<32>::kThreads : kSmallThreads);
        cfg.dynamicSmemBytes = tiny == 16 ? Tiny<16>::smem(longest) : tiny == 32 ? Tiny<32>::smem(longest)
                                                                                : 1024 + (2 * per + 8) * kBlkBytes + (cluster > 1 ? 4 * kTileF : 0);
        cfg.stream = ctx.stream;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)cluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        at[1] = overlap();
        cfg.attrs = at;
        cfg.numAttrs = beside && b == 0 ? 2 : 1;
        if (cudaLaunchKernelEx(&cfg, kernel, J) != cudaSuccess) return cuda_error();
    }
    return CF_OK;
}

// The cooperative launch.
struct Coop {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    Coop(const LaunchCtx& ctx, bool pair) {
        cfg.gridDim = dim3((unsigned)(pair ? ctx.num_sms / 2 * 2 : ctx.num_sms));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cfg.stream = ctx.stream;
        at[0].id = cudaLaunchAttributeCooperative;
        at[0].val.cooperative = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = 2;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = pair ? 2 : 1;
    }
    Coop(const Coop&) = delete;
};

// Whether the device holds all of the cooperative launch's blocks at once, asked once for each device: a call that finds out at the
// launch has taken its momentum steps by then.
bool coop_fits(const LaunchCtx& ctx, bool pair) {
    constexpr int kDevices = 64;
    static std::atomic<int8_t> known[2][kDevices];  // 0: not asked, 1: fits, -1: does not
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    int8_t k = known[pair][dev].load(std::memory_order_relaxed);
    if (k == 0) {
        int have = 0;
        Coop coop(ctx, pair);
        const cudaError_t e =
            pair ? cudaOccupancyMaxActiveClusters(&have, ns_kernel<true>, &coop.cfg)
                 : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&have, ns_kernel<false>, kThreads, kSmem);
        if (e != cudaSuccess) return false;
        k = have >= (pair ? ctx.num_sms / 2 : 1) ? 1 : -1;
        known[pair][dev].store(k, std::memory_order_relaxed);
    }
    return k > 0;
}

// uniform: the matrices are of one batch, a matrix apart.  few: what take_few took out of a list.
cf_status run(const LaunchCtx& ctx, const Poly& p, float mu, int nesterov, std::vector<Mat>& mats, std::vector<Mat>& few, void* ws,
              bool uniform) {
    const int cluster = cluster_of(mats);
    if (cluster == 0) {
        if (cudaFuncSetAttribute(ns_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess ||
            cudaFuncSetAttribute(ns_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
            return cuda_error();
        for (size_t b = 0; b < mats.size(); b += kMaxMats)
            if (!coop_fits(ctx, plan_sizes(&mats[b], (int)std::min<size_t>(kMaxMats, mats.size() - b)))) return cuda_error();
    }
    if (!few.empty())
        if (const cf_status st = (few.size() == 1 ? run_small<1> : run_small<kMaxMats>)(ctx, p, mu, nesterov, few, 1, false, false); st != CF_OK)
            return st;
    if (cluster)
        return (uniform || mats.size() == 1 ? run_small<1> : run_small<kMaxMats>)(ctx, p, mu, nesterov, mats, cluster, uniform, !few.empty());
    for (size_t b = 0; b < mats.size(); b += kMaxMats) {
        Job J{};
        J.count = (int)std::min<size_t>(kMaxMats, mats.size() - b);
        const bool pair = plan_sizes(&mats[b], J.count);
        place(&mats[b], J.count, pair, static_cast<char*>(ws), &J.part);
        J.share = gram_share(&mats[b], J.count, pair, &J.half_g);
        J.uw = pair ? 4 : update_width(&mats[b], J.count);
        for (int i = 0; i < J.count; ++i) {
            Mat& M = J.mat[i] = mats[b + i];
            M.ut = (M.nx + J.uw - 1) / J.uw;
            M.n0 = J.nn, M.c0 = J.nc, M.s0 = J.ns, M.u0 = J.nu, M.b0 = J.blocks;
            const int tiles = M.gt * (M.gt + 1) / 2;
            J.nn += M.chunks;
            J.nc += M.rb * M.cb;
            J.blocks += tiles * M.nx;
            J.ns += tiles;
            J.nu += M.gt * M.ut;
        }
        // the other side's columns in halves where there are then items enough for one round; U's last round too
        const int units = kPlanSms / (pair ? 2 : 1), left = J.nu % units;
        J.half = 2 * J.ns <= units;
        J.whole = J.nu - (2 * left <= units ? left : 0);
        if (J.share) list_cuts(J);
        J.steps = p.steps, J.a = p.a, J.b = p.b, J.c = p.c, J.eps = p.eps, J.cap = cap_of(p), J.mu = mu, J.nesterov = nesterov;
        J.sync = static_cast<uint32_t*>(ws);
        J.status = ctx.status;
        J.wait_ns = ctx.wait_ns;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)J.nn);
        cfg.blockDim = dim3(256);
        cfg.stream = ctx.stream;
        cudaLaunchAttribute at = overlap();
        cfg.attrs = &at;
        cfg.numAttrs = !few.empty() && b == 0 ? 1 : 0;
        if (cudaLaunchKernelEx(&cfg, ns_input_kernel, J) != cudaSuccess) return cuda_error();
        cfg.gridDim = dim3((unsigned)J.nc);
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, ns_convert_kernel, J) != cudaSuccess) return cuda_error();
        Coop coop(ctx, pair);
        if (cudaLaunchKernelEx(&coop.cfg, pair ? ns_kernel<true> : ns_kernel<false>, J) != cudaSuccess) return cuda_error();
    }
    return CF_OK;
}

std::vector<Mat> batch_of(const cf_ns_desc* d, const void* g, uint16_t* o) {
    std::vector<Mat> mats((size_t)d->batch);
    const int f32 = d->dtype == CF_DT_F32;
    const int64_t count = d->rows * d->cols;
    for (int64_t i = 0; i < d->batch; ++i) {
        mats[i].rows = d->rows, mats[i].cols = d->cols, mats[i].f32 = f32;
        mats[i].g = static_cast<const char*>(g) + i * count * (f32 ? 4 : 2);
        mats[i].o = o + i * count;
    }
    return mats;
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

size_t cf_orthogonalize_workspace_size(const cf_ns_desc* desc) try {
    if (ns_check(desc) != CF_OK) return 0;
    std::vector<Mat> mats = batch_of(desc, nullptr, nullptr);
    return workspace_of(mats);
} catch (const std::bad_alloc&) {  // the list of matrices
    return 0;
}

cf_status cf_orthogonalize(const cf_ns_desc* desc, const void* g, uint16_t* o, void* ws, size_t ws_bytes, void* stream) try {
    if (const cf_status st = ns_check(desc); st != CF_OK) return st;
    if (g == nullptr || o == nullptr || !aligned16(g) || !aligned16(o) || !aligned16(ws)) return CF_ERR_INVALID_ARG;
    std::vector<Mat> mats = batch_of(desc, g, o);
    if (ws == nullptr || ws_bytes < workspace_of(mats)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    std::vector<Mat> none;
    return run(ctx, Poly{desc->steps, desc->a, desc->b, desc->c, desc->eps}, 0.f, 0, mats, none, ws, true);
} catch (const std::bad_alloc&) {  // the list of matrices
    return CF_ERR_UNSUPPORTED;
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

static std::vector<Mat> list_of(int32_t count, const cf_muon_param* p) {
    std::vector<Mat> mats((size_t)count);
    for (int32_t i = 0; i < count; ++i) {
        Mat& M = mats[i];
        M.g = p[i].g, M.m = p[i].m, M.w = p[i].w, M.o = p[i].w_bf16;
        M.rows = p[i].rows, M.cols = p[i].cols, M.f32 = 1;
    }
    return mats;
}

size_t cf_muon_workspace_size(int32_t count, const cf_muon_param* params) try {
    if (count == 0 || muon_check(count, params) != CF_OK) return 0;
    std::vector<Mat> mats = list_of(count, params);
    take_few(mats);
    return workspace_of(mats);
} catch (const std::bad_alloc&) {  // the list of matrices
    return 0;
}

cf_status cf_muon_step(int32_t count, const cf_muon_param* params, const cf_muon_hyper* h, void* ws, size_t ws_bytes,
                       void* stream) try {
    if (h == nullptr) return CF_ERR_INVALID_ARG;
    const Poly p{h->steps, h->a, h->b, h->c, h->eps};
    if (!poly_ok(p) || !std::isfinite(h->lr) || !std::isfinite(h->momentum) || !std::isfinite(h->weight_decay))
        return CF_ERR_INVALID_ARG;
    if (const cf_status st = muon_check(count, params); st != CF_OK) return st;
    if (!aligned16(ws)) return CF_ERR_INVALID_ARG;
    if (h->steps > 16) return CF_ERR_UNSUPPORTED;
    if (count == 0) return CF_OK;
    std::vector<Mat> mats = list_of(count, params);
    for (int32_t i = 0; i < count; ++i) {
        mats[i].keep = 1.f - h->lr * h->weight_decay;
        mats[i].step = h->lr * params[i].scale;
    }
    std::vector<Mat> few = take_few(mats);
    if (ws == nullptr || ws_bytes < workspace_of(mats)) return CF_ERR_WORKSPACE;
    LaunchCtx ctx;
    if (!cf_device_ctx(&ctx, stream)) return CF_ERR_CUDA;
    return run(ctx, p, h->momentum, h->nesterov != 0, mats, few, ws, false);
} catch (const std::bad_alloc&) {  // the list of matrices
    return CF_ERR_UNSUPPORTED;
}

}  // extern "C"
