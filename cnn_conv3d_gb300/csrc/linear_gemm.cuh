// linear_gemm.cuh -- the product of linear.cu on the tensor cores: D [m][n] = sum over K of A [m][K] B [n][K] with an epilogue,
// one kernel template for the three directions, instantiated by a translation unit each.
//
//   forward          A = x [rows][k],       B = w [n][k]                both with the contracted axis contiguous (K-major)
//   backward data    A = dz [rows][n],      B = w as [K = n][k]         B with its rows contiguous (MN-major)
//   backward weight  A = dz as [K = rows][n], B = x as [K = rows][k]    both MN-major
// or the two exchanged (SWAP) where that side is narrow: few rows in the forward and the backward data, so that the weights' rows
// fill the 128 lanes of a tile and the rows are its columns, and a narrow k in the backward weight.
//
// A CTA is a TMA warp, an issuing thread and sixteen epilogue warps (eight, see below).  Operands come in stages of 64 of the contracted
// axis (128-byte rows, swizzled); tiles are 128 rows by up to 256 columns, or 256 by 256 on a pair of CTAs with one instruction for both, each CTA
// fetching half of either side: then a stage costs 64 bytes of L2 a cycle and SM, where a lone CTA's would cost 96 of the about 70
// that it gives.  The accumulator is double: the epilogue of a tile runs under the products of the next.
//
// The tensor cores cut off what an fp32 sum cannot hold: about 1.7e-8 of the result for each step of 16 of the contracted axis where
// the values' signs are mixed (weights of 2048 x 8192 from 16384 rows: 1.7e-5 off, where sums in fp32 that round are 1.4e-6).  Where the
// result is fp32 they therefore sum 24 blocks of the axis at a time, and the epilogue warps, then eight with the registers for it, add
// these sums up, rounding, under the next blocks' products (SUMS): 1.5e-6, and 393 us in place of 362; 16 blocks took 406, 32 390.
// Bias gradients likewise, a thread or a lane to each: of rows whose sizes differ by e^3 each way 1.5e-5 and 1.8e-5 off (16384 rows of 4096,
// 20000 of 38912) with one sum over all of a tile's rows, 5e-7 so, at the same times.
//
// Where there are fewer tiles than CTAs, a cluster may take each, its CTAs even shares of the contracted axis, whose sums they add up
// through distributed shared memory, each CTA of some columns (linear_split_kernel).  Otherwise
// tiles are dealt out whole, and what is left over for a last, uneven round (or all of it, where there are fewer tiles than CTAs) in
// even shares of 64-blocks of the contracted axis; tiles that are cut leave fp32 parts, joined in order by a second launch.
#pragma once

#include <type_traits>

#include "cf_internal.h"
#include "cf_pair.cuh"
#include "cf_two.cuh"

namespace cf {

enum { OP_FWD = CF_LINEAR_FWD, OP_DGRAD = CF_LINEAR_DGRAD, OP_WGRAD = CF_LINEAR_WGRAD };

// What the epilogue needs.  Rows and columns are the output's, not the tile's, whatever SWAP.
struct LinEpi {
    const float* bias;
    const void* add;         // forward: residual
    const uint16_t* pre_in;  // backward data: the derivative's argument
    uint16_t* pre_out;       // forward
    void* out;
    float* db;               // backward weight: sums of dz's rows, or NULL
    int64_t pitch, rows;
    int cols;
    int act, f32, accumulate;
    float slope, scale;
};

// The epilogue's way to rows in memory: a warp's 32 rows x `gw` columns pass through shared memory (128-byte rows, swizzled, in
// slabs of 4 KB), from and to which TMA copies them.  A lane owns a row, so that its own accesses to memory would be 32 lines an
// instruction: stores that way took the data pipe 57 cycles a kilobyte and 64 -> 256 on 2.1M voxels 731 us.
struct LinStage {
    int tma;                   // rows begin and end at 16 bytes; otherwise a warp copies value by value along the rows
    int gw;                    // columns of a pass: 64, or 32 of fp32 with no pre-activation beside them
    int sets, turns;           // sets of epilogue warps that take the tiles in turn; a set's warps for each quarter of the lanes
    int out_bytes, aux_bytes;  // a warp's room: the output (and what is added to it, in the same place), the pre-activation
    int load_add, load_aux;
};

struct LinGemm {
    LinStage st;
    int64_t m, n;            // D's sizes
    int nkb;                 // 64-blocks of the contracted axis
    int tm, tn;              // tiles
    int bn;                  // columns of a tile
    int sub;                 // a narrow tile has so many times 128 rows, side by side in the accumulator
    int a_mn, b_mn;          // operands with their rows contiguous
    int a_box, b_box;        // K-major: rows of a copy
    int stages, stage_bytes;
    int whole;               // tiles that are dealt out whole
    int share;               // a unit's blocks of the others
    int64_t rest;            // all blocks of the others
    int units;               // CTAs or pairs
    int seg;                 // SUMS: blocks that the tensor cores sum
    int split;               // CTAs of a cluster that share a tile (linear_split_kernel), or 0
    float *part, *dpart;     // parts of cut tiles: a unit's two slots of 128 x bn values a CTA; of db, 256 values a slot
    int* status;
    uint64_t wait_ns;
};

constexpr int kLinEpiWarps = 16;
constexpr int kLinSumWarps = 8;  // with SUMS
constexpr int threads_of_linear(bool sums) { return 64 + 32 * (sums ? kLinSumWarps : kLinEpiWarps); }
constexpr int kLinMostStages = 10;
constexpr uint32_t kLinOnes = 16 << 10;             // 128 rows of 64 ones (backward weight)
constexpr uint32_t kLinSmem = 232448;               // all of it: ones, passes and stages, then LinShared
constexpr uint32_t kLinBias = 64 * 4;               // of a warp's pass

// ------------------------------------------------------------------------------------------------------------------ activations
constexpr float kGeluA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float t) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
    return r;
}
__device__ __forceinline__ float rcp(float t) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
    return r;
}
// 1 / (1 + 2^t)
__device__ __forceinline__ uint64_t gate2(uint64_t t) {
    float a, b;
    apart(t, a, b);
    apart(add2(two(ex2(a), ex2(b)), two(1.f, 1.f)), a, b);
    return two(rcp(a), rcp(b));
}
// 1 / (1 + exp(-t)), t = z for SiLU, kGeluA (z + kGeluB z^3) for GELU; infinities give 0 and 1.
__device__ __forceinline__ uint64_t silu_gate(uint64_t z) { return gate2(mul2(z, two(-kLog2e, -kLog2e))); }
__device__ __forceinline__ uint64_t gelu_gate(uint64_t z) {
    constexpr float a = -kLog2e * kGeluA, b = -kLog2e * kGeluA * kGeluB;
    return gate2(mul2(z, fma2(mul2(z, z), two(b, b), two(a, a))));
}
// z within +-100, where the derivatives are 1 and 0 already and no product of theirs is inf times 0; a NaN stays.
__device__ __forceinline__ float bounded(float z) {
    asm("{min.NaN.f32 %0, %0, 0f42C80000;\n\tmax.NaN.f32 %0, %0, 0fC2C80000;}" : "+f"(z));
    return z;
}
__device__ __forceinline__ uint64_t smooth_grad(int act, uint64_t z) {
    float a, b;
    apart(z, a, b);
    z = two(bounded(a), bounded(b));
    const uint64_t e = act == CF_ACT_SILU ? silu_gate(z) : gelu_gate(z);
    uint64_t t = mul2(mul2(z, e), fma2(e, two(-1.f, -1.f), two(1.f, 1.f)));
    if (act == CF_ACT_GELU) {
        constexpr float c = 3.f * kGeluA * kGeluB;
        t = mul2(t, fma2(mul2(z, z), two(c, c), two(kGeluA, kGeluA)));
    }
    return add2(e, t);
}
// The activation of all, with one branch.
template <int N>
__device__ __forceinline__ void activate(const LinEpi& E, float (&v)[N]) {
    if (E.act == CF_ACT_LRELU) {
        if (E.slope == 1.f) return;
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = v[e] > 0.f ? v[e] : E.slope * v[e];
        return;
    }
    const bool silu = E.act == CF_ACT_SILU;
    constexpr int kStep = N > 1 ? 2 : 1;
#pragma unroll
    for (int e = 0; e < N; e += kStep) {
        const uint64_t z = two(v[e], v[e + kStep - 1]);
        apart(mul2(z, silu ? silu_gate(z) : gelu_gate(z)), v[e], v[e + kStep - 1]);
    }
}
template <int N>
__device__ __forceinline__ void times_grad(const LinEpi& E, const float (&z)[N], float (&v)[N]) {
    if (E.act == CF_ACT_LRELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] *= z[e] > 0.f ? 1.f : E.slope;
        return;
    }
    const int act = E.act;
    constexpr int kStep = N > 1 ? 2 : 1;
#pragma unroll
    for (int e = 0; e < N; e += kStep)
        apart(mul2(two(v[e], v[e + kStep - 1]), smooth_grad(act, two(z[e], z[e + kStep - 1]))), v[e], v[e + kStep - 1]);
}

// --------------------------------------------------------------------------------------------------------- rows of the epilogue
// Byte `at` of row r (at most 64 fp32 columns) in a buffer of slabs.
__device__ __forceinline__ uint32_t slab_at(int r, int at) { return (at >> 7) * 4096 + r * 128 + ((((at & 127) >> 4) ^ (r & 7)) << 4) + (at & 15); }

// 16 columns of the thread's row from column c of the pass on.
__device__ __forceinline__ void slab_load16(const uint8_t* buf, int f32, int r, int c, float (&v)[16]) {
    if (f32) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const float4 q = *reinterpret_cast<const float4*>(buf + slab_at(r, 4 * (c + e)));
            v[e] = q.x, v[e + 1] = q.y, v[e + 2] = q.z, v[e + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
            const uint4 q = *reinterpret_cast<const uint4*>(buf + slab_at(r, 2 * (c + e)));
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) v[e + 2 * x] = __uint_as_float(u[x] << 16), v[e + 2 * x + 1] = __uint_as_float(u[x] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ void slab_store16(uint8_t* buf, int f32, int r, int c, const float (&v)[16]) {
    if (f32) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(buf + slab_at(r, 4 * (c + e))) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < 16; e += 8)
            *reinterpret_cast<uint4*>(buf + slab_at(r, 2 * (c + e))) =
                make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]), pack_bf16x2(v[e + 4], v[e + 5]), pack_bf16x2(v[e + 6], v[e + 7]));
    }
}
// A warp's copies between a buffer and rows that begin anywhere: rows [i, i + 32) of `rows`, columns [j, j + width) of `cols`; eight
// accesses of a lane in flight.  (Words of two bf16 values, put together from neighbouring lanes' where a row begins inside one, took
// the backward data 515 -> 130 of 100003 rows 208 us, in place of 68.)
template <bool IN, bool ALL, typename T>
__device__ __forceinline__ void slab_columns(uint8_t* buf, T* at, int high, int c, int64_t pitch) {
    int to[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) to[r] = slab_at(r, (int)sizeof(T) * c);
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += 8, buf += 1024) {
        T v[8];
        T* from = at;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (!IN)
                v[r] = *reinterpret_cast<const T*>(buf + to[r]);
            else
                v[r] = ALL || r0 + r < high ? *from : T(0);
            from += pitch;
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (IN)
                *reinterpret_cast<T*>(buf + to[r]) = v[r];
            else if (ALL || r0 + r < high)
                *at = v[r];
            at += pitch;
        }
    }
}
template <bool IN, typename T>
__device__ __forceinline__ void slab_copy(uint8_t* buf, T* p, int64_t i, int64_t rows, int j, int cols, int width, int64_t pitch) {
    const int lane = threadIdx.x & 31, high = (int)min((int64_t)32, rows - i);
    for (int c = lane; c < width && j + c < cols; c += 32) {
        T* at = p + i * pitch + j + c;
        if (high == 32)
            slab_columns<IN, true>(buf, at, high, c, pitch);
        else
            slab_columns<IN, false>(buf, at, high, c, pitch);
    }
}
template <bool IN>
__device__ __forceinline__ void slab_copy(uint8_t* buf, void* p, int f32, int64_t i, int64_t rows, int j, int cols, int width, int64_t pitch) {
    if (f32)
        slab_copy<IN>(buf, static_cast<float*>(p), i, rows, j, cols, width, pitch);
    else
        slab_copy<IN>(buf, static_cast<uint16_t*>(p), i, rows, j, cols, width, pitch);
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m), "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// 16 columns of a row from column c of the pass on: the pass's bias, what is added and the derivative's argument are in shared memory.
template <int OP>
__device__ __forceinline__ void finish_row(const LinEpi& E, const LinStage& S, uint8_t* out, uint8_t* aux, const float* bias, int r, int c, float (&v)[16]) {
    float t[16];
    if (OP == OP_FWD) {
        if (E.bias) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 q = *reinterpret_cast<const float4*>(bias + c + e);
                apart(add2(two(v[e], v[e + 1]), two(q.x, q.y)), v[e], v[e + 1]);
                apart(add2(two(v[e + 2], v[e + 3]), two(q.z, q.w)), v[e + 2], v[e + 3]);
            }
        }
        if (S.aux_bytes) slab_store16(aux, 0, r, c, v);
        activate(E, v);
    } else if (OP == OP_DGRAD && S.load_aux) {
        slab_load16(aux, 0, r, c, t);
        times_grad(E, t, v);
    }
    if (S.load_add) {
        slab_load16(out, E.f32, r, c, t);
#pragma unroll
        for (int e = 0; e < 16; e += 2) apart(fma2(two(v[e], v[e + 1]), two(E.scale, E.scale), two(t[e], t[e + 1])), v[e], v[e + 1]);
    } else if (E.scale != 1.f) {
#pragma unroll
        for (int e = 0; e < 16; e += 2) apart(mul2(two(v[e], v[e + 1]), two(E.scale, E.scale)), v[e], v[e + 1]);
    }
    slab_store16(out, E.f32, r, c, v);
}
// N rows of column j from row i on (neighbouring threads have neighbouring columns).
template <int OP, int N>
__device__ __forceinline__ void finish_column(const LinEpi& E, int64_t i, int j, float (&v)[N]) {
    if (j >= E.cols) return;
    const int cnt = (int)min((int64_t)N, E.rows - i);
    const int64_t o = i * E.pitch + j;
    float t[N];
    auto load = [&](const void* p, int f32) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            t[e] = e >= cnt ? 0.f
                   : f32    ? static_cast<const float*>(p)[o + e * E.pitch]
                            : bf16_bits_to_float(static_cast<const uint16_t*>(p)[o + e * E.pitch]);
    };
    if (OP == OP_FWD) {
        const float b = E.bias ? E.bias[j] : 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            v[e] += b;
            if (E.pre_out && e < cnt) E.pre_out[o + e * E.pitch] = __bfloat16_as_ushort(__float2bfloat16_rn(v[e]));
        }
        activate(E, v);
    } else if (OP == OP_DGRAD && E.pre_in) {
        load(E.pre_in, 0);
        times_grad(E, t, v);
    }
    const void* add = OP == OP_WGRAD ? (E.accumulate ? E.out : nullptr) : E.add;
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = 0.f;
    if (add) load(add, E.f32);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float r = add ? fmaf(E.scale, v[e], t[e]) : E.scale * v[e];
        if (e < cnt) {
            if (E.f32)
                static_cast<float*>(E.out)[o + e * E.pitch] = r;
            else
                static_cast<uint16_t*>(E.out)[o + e * E.pitch] = __bfloat16_as_ushort(__float2bfloat16_rn(r));
        }
    }
}

// ------------------------------------------------------------------------------------------------------------------------- work
struct LinItem {
    int mt, nt, kb0, kb1;
    int slot;  // where a part goes, -1 for a whole tile
};
// Tiles in bands of eight rows of tiles, so that what runs at one time shares operands in L2.
__device__ __forceinline__ void tile_of(const LinGemm& G, int t, int& mt, int& nt) {
    const int band = t / (8 * G.tn), r = t - band * 8 * G.tn, high = min(8, G.tm - 8 * band);
    nt = r / high;
    mt = 8 * band + r - nt * high;
}
struct LinWalk {
    int t, e, kb, left;  // the next whole tile; the next of the others, its block, and how many the unit still takes
    __device__ __forceinline__ LinWalk(const LinGemm& G, int unit) : t(unit), e(0), kb(0), left(0) {
        const int64_t at = (int64_t)unit * G.share;
        if (at >= G.rest) return;
        e = (int)(at / G.nkb), kb = (int)(at - (int64_t)e * G.nkb);
        left = (int)min((int64_t)G.share, G.rest - at);
    }
    __device__ __forceinline__ bool next(const LinGemm& G, int unit, LinItem& s) {
        if (t < G.whole) {
            tile_of(G, t, s.mt, s.nt);
            s.kb0 = 0, s.kb1 = G.nkb, s.slot = -1;
            t += G.units;
            return true;
        }
        if (left == 0) return false;
        tile_of(G, G.whole + e, s.mt, s.nt);
        const int take = min(left, G.nkb - kb);
        s.kb0 = kb, s.kb1 = kb + take;
        s.slot = take == G.nkb ? -1 : 2 * unit + (kb == 0);
        left -= take, kb = 0, ++e;
        return true;
    }
};

struct LinShared {
    uint64_t full[kLinMostStages], empty[kLinMostStages], tfull[2], tempty[2], in[kLinEpiWarps], drain;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(LinShared) % 16 == 0, "the bias is before it");
// The accumulators in turn, and how often each has been filled.
struct Accumulators {
    uint32_t uses[2] = {0, 0};
    int flip = 0;
    __device__ __forceinline__ int next(bool sums) const { return sums ? 0 : flip; }
    __device__ __forceinline__ void used(int acc, bool sums) {
        ++uses[acc];
        if (!sums) flip ^= 1;
    }
};
struct LinRing {
    int stage = 0;
    uint32_t bits = 0, issued = 0;
    __device__ __forceinline__ uint32_t parity() const { return (bits >> stage) & 1; }
    __device__ __forceinline__ void next(int stages) {
        bits ^= 1u << stage;
        if (++stage == stages) stage = 0;
    }
};

// The sums of dz's rows come from products with ones: they are taken with the first tile across the other side, into the second
// accumulator, while all of the tile's own products go to the first.
template <int OP, bool SWAP>
__device__ __forceinline__ bool takes_sums(const LinEpi& E, const LinItem& s) {
    return OP == OP_WGRAD && E.db && (SWAP ? s.mt : s.nt) == 0;
}

// Rows of a tile's parts of 128 (of one CTA) that there are.
template <bool PAIR>
__device__ __forceinline__ int parts_of(const LinGemm& G, const LinItem& s) {
    return PAIR || G.sub == 1 ? 1 : (int)min((int64_t)G.sub, (G.m - (int64_t)s.mt * 128 * G.sub + 127) / 128);
}
// The passes of an epilogue warp over the tiles that it finishes itself, in the order that it takes them: of two sets, those whose
// accumulator is the set's, by the rule of all other warps (a tile that takes sums turns the accumulators no further).
template <int OP, bool SWAP, bool PAIR>
struct LinPasses {
    LinWalk way;
    LinItem s;
    int pass, part, c, local;  // pass of the tile: its 128 rows, and first column; the unit's tiles so far that turned the accumulators
    bool more;
    __device__ __forceinline__ LinPasses(const LinGemm& G, const LinEpi& E, int unit, int set, int turn) : way(G, unit), pass(1 << 20), local(0), more(true) {
        next(G, E, unit, set, turn);
    }
    __device__ __forceinline__ void next(const LinGemm& G, const LinEpi& E, int unit, int set, int turn) {
        const int across = (G.bn + G.st.gw - 1) / G.st.gw;
        pass += G.st.turns;
        while (more && (pass >= 1 << 20 || pass >= across * parts_of<PAIR>(G, s))) {
            bool mine;
            do {
                more = way.next(G, unit, s);
                const bool sums = takes_sums<OP, SWAP>(E, s);
                mine = s.slot < 0 && (G.st.sets == 1 || (sums ? 0 : local & 1) == set);  // Accumulators::next
                if (!sums) ++local;
            } while (more && !mine);
            pass = turn;
        }
        part = pass / across;
        c = (pass - part * across) * G.st.gw;
    }
};

struct LinMaps {
    CUtensorMap a, b;      // operands
    CUtensorMap out, add;  // the output's rows and what is added
    CUtensorMap aux;       // the pre-activation
};

// TMA: S.tma, which a kernel of both would pay for with registers.
template <bool PAIR, int OP, bool SWAP, bool TMA, bool SUMS>
__global__ void __launch_bounds__(threads_of_linear(SUMS), 1) linear_gemm_kernel(const __grid_constant__ LinMaps M, const __grid_constant__ LinGemm G,
                                                                     const __grid_constant__ LinEpi E) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    constexpr int kLinThreads = threads_of_linear(SUMS);
    if (smem_u32(smem_raw) & 1023) {  // the swizzle goes by the address, and there is no room to move in
        if (threadIdx.x == 0) atomicCAS(G.status, 0, (int)WAIT_PROBE);
        return;
    }
    uint8_t* ones = smem_raw;
    LinShared& sh = *reinterpret_cast<LinShared*>(smem_raw + kLinSmem - sizeof(LinShared));
    uint8_t* passes = ones + (OP == OP_WGRAD ? kLinOnes : 0);
    uint8_t* ring = passes + (SWAP ? 0 : 4 * G.st.sets * G.st.turns * (G.st.out_bytes + G.st.aux_bytes));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = PAIR ? (int)cluster_rank() : 0;
    const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x;
    if (warp == 0) {
        // a lane to each barrier
        if (lane == 0) {
            tma_prefetch_desc(&M.a);
            tma_prefetch_desc(&M.b);
            sh.abort = 0;
        }
        if (lane < kLinMostStages) {
            mbar_init(&sh.full[lane], PAIR && rank == 0 ? 2 : 1);
            mbar_init(&sh.empty[lane], 1);
        } else if (lane < kLinMostStages + 2) {
            mbar_init(&sh.tfull[lane - kLinMostStages], 1);
            mbar_init(&sh.tempty[lane - kLinMostStages], (PAIR ? 2 : 1) * 4 * G.st.turns);
        } else if (lane == kLinMostStages + 2) {
            mbar_init(&sh.drain, 1);
        }
        if (lane >= 32 - kLinEpiWarps) mbar_init(&sh.in[lane - (32 - kLinEpiWarps)], 1);
        fence_barrier_init();
        __syncwarp();
    }
    if (OP == OP_WGRAD) {
        for (int e = threadIdx.x; e < (int)kLinOnes / 4; e += kLinThreads) reinterpret_cast<uint32_t*>(ones)[e] = 0x3F803F80u;
        fence_proxy_async_smem();
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
    // the barriers are the first warp's own, so that a lone CTA's loads need not wait for the others
    if (PAIR)
        cluster_sync();
    else if (warp == 0)
        asm volatile("bar.arrive 1, %0;" ::"n"(kLinThreads) : "memory");
    else
        named_bar_sync(1, kLinThreads);
    tc_fence_after();
    // begun under the end of the launch before.  (Letting the joining launch begin under this one's end took 1.3 us longer.)
    asm volatile("griddepcontrol.wait;" ::: "memory");

    LinWalk way(G, unit);
    LinItem s;
    LinRing R;
    if (warp == 0) {
        // a lane for each copy of a stage: one of A's (two where it is MN-major), the others of B's
        const int bhalf = PAIR ? G.bn / 2 : G.bn;
        const bool isb = lane >= 2;
        const int q = isb ? lane - 2 : lane;
        bool ok = true;
        while (ok && way.next(G, unit, s)) {
            int64_t m0 = (int64_t)s.mt * (PAIR ? 256 : 128 * G.sub) + 128 * rank;
            const int64_t n0 = (int64_t)s.nt * G.bn + bhalf * rank;
            const int parts = parts_of<PAIR>(G, s);
            const int na = G.a_mn ? (int)min((int64_t)2, max((int64_t)0, (G.m - m0 + 63) / 64)) : 1;
            const int nb = G.b_mn ? (int)min((int64_t)(bhalf + 63) / 64, max((int64_t)0, (G.n - n0 + 63) / 64)) : 1;
            const uint32_t bytes = (G.a_mn ? na * 8192 : 16384) + (G.b_mn ? nb * 8192 : G.b_box * 128);
            const bool mn = isb ? G.b_mn : G.a_mn, mine = q < (isb ? nb : na);
            const uint32_t dst = (isb ? 16384 : 0) + q * 8192;
            const CUtensorMap* map = isb ? &M.b : &M.a;
            for (int part = 0; ok && part < parts; ++part, m0 += 128) {
                const int64_t r0 = isb ? n0 : m0;
                for (int kb = s.kb0; kb < s.kb1; ++kb) {
                    ok = __all_sync(~0u, mbar_wait(&sh.empty[R.stage], R.parity() ^ 1, &sh.abort, G.wait_ns, G.status, WAIT_PRODUCER_EMPTY));
                    if (!ok) break;
                    uint64_t* bar = &sh.full[R.stage];
                    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                    __syncwarp();
                    if (mine) {
                        uint8_t* to = ring + R.stage * G.stage_bytes + dst;
                        if (mn)
                            tma_load_2d(to, map, bar, (int)(r0 + 64 * q), (int)(64 * kb));
                        else
                            tma_load_2d(to, map, bar, (int)(64 * kb), (int)r0);
                    }
                    R.issued |= 1u << R.stage;
                    R.next(G.stages);
                }
            }
        }
    } else if (warp == 1 && lane == 0) {
        const bool second = PAIR && rank == 1;
        const uint32_t idesc = idesc_bf16(PAIR ? 256 : 128, G.bn, G.a_mn, G.b_mn);
        // A's rows times ones [K][N]: 16 (32 for a pair) equal columns; exchanged, ones [128][K] times B: equal rows
        const uint32_t idesc1 = SWAP ? idesc_bf16(128, G.bn, 0, G.b_mn) : idesc_bf16(PAIR ? 256 : 128, PAIR ? 32 : 16, G.a_mn, 0);
        const uint64_t one = sdesc(smem_u32(ones), 16, 1024, SWZ_128B);
        const uint32_t astep = G.a_mn ? 2048 : 32, bstep = G.b_mn ? 2048 : 32;
        const uint32_t alead = G.a_mn ? 8192 : 16, blead = G.b_mn ? 8192 : 16;
        Accumulators A;
        bool alone = false;  // the tile before took sums
        bool ok = true;
        auto free_of = [&](int acc) {
            return A.uses[acc] == 0 || mbar_wait(&sh.tempty[acc], (A.uses[acc] - 1) & 1, &sh.abort, G.wait_ns, G.status, WAIT_MMA_TMEM_EMPTY);
        };
        while (ok && way.next(G, unit, s)) {
            if (second) {
                for (int kb = s.kb0; ok && kb < s.kb1; ++kb) {
                    ok = mbar_wait(&sh.full[R.stage], R.parity(), &sh.abort, G.wait_ns, G.status, WAIT_MMA_FULL);
                    if (!ok) break;
                    arrive_first(&sh.full[R.stage]);
                    R.next(G.stages);
                }
                continue;
            }
            const bool sums = takes_sums<OP, SWAP>(E, s);
            if (sums || alone) ok = free_of(0) && free_of(1);
            alone = sums;
            const int parts = parts_of<PAIR>(G, s), seg = SUMS ? G.seg : s.kb1 - s.kb0;
            for (int k0 = s.kb0; ok && k0 < s.kb1; k0 += seg) {
                const int acc = A.next(sums), k1 = min(k0 + seg, s.kb1);
                const uint32_t d = sh.tmem + acc * 256, d1 = sh.tmem + 256;
                ok = free_of(acc);
                tc_fence_after();
                for (int part = 0; ok && part < parts; ++part) {
                    const uint32_t dp = d + part * G.bn;
                    for (int kb = k0; ok && kb < k1; ++kb) {
                        ok = mbar_wait(&sh.full[R.stage], R.parity(), &sh.abort, G.wait_ns, G.status, WAIT_MMA_FULL);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t as = smem_u32(ring + R.stage * G.stage_bytes), bs = as + 16384;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint64_t ad = sdesc(as + k * astep, alead, 1024, SWZ_128B), bd = sdesc(bs + k * bstep, blead, 1024, SWZ_128B);
                            const uint32_t more = kb > k0 || k > 0;
                            if (PAIR)
                                umma_pair(dp, ad, bd, idesc, more);
                            else
                                umma_bf16(dp, ad, bd, idesc, more);
                            if (OP == OP_WGRAD && sums) {
                                if (PAIR)
                                    umma_pair(d1, ad, one, idesc1, more);
                                else
                                    umma_bf16(d1, SWAP ? one : ad, SWAP ? bd : one, idesc1, more);
                            }
                        }
                        if (PAIR)
                            commit_pair(&sh.empty[R.stage]);
                        else
                            umma_commit(&sh.empty[R.stage]);
                        R.next(G.stages);
                    }
                }
                if (!ok) break;
                if (PAIR)
                    commit_pair(&sh.tfull[acc]);
                else
                    umma_commit(&sh.tfull[acc]);
                A.used(acc, sums);
            }
        }
    } else if (warp >= 2) {
        // a pass of columns at a time, a set's warps of a quarter of the lanes in turn, 16 columns of the thread's lane at once
        const LinStage& S = G.st;
        const int q = warp & 3, group = (warp - 2) >> 2, set = S.turns == 4 ? 0 : group >> 1, turn = S.turns == 4 ? group : group & 1;
        const int r = 32 * q + lane;
        uint8_t *out = passes + (warp - 2) * (S.out_bytes + S.aux_bytes), *aux = out + S.out_bytes;
        const uint32_t in_bytes = SWAP || !TMA ? 0 : (S.load_add ? S.out_bytes : 0) + (S.load_aux ? S.aux_bytes : 0);
        uint32_t done = 0, asked = 0;  // passes finished, and those whose loads were issued
        bool ok = set < S.sets;
        LinPasses<OP, SWAP, PAIR> ahead(G, E, unit, set, turn);
        // the next pass's loads, once the present one's store has been read
        auto ask = [&]() {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
            if (!in_bytes || !ahead.more) return;
            if (lane == 0) {
                const int row = ahead.s.mt * (PAIR ? 256 : 128 * G.sub) + 128 * (rank + ahead.part) + 32 * q, col = ahead.s.nt * G.bn + ahead.c;
                mbar_arrive_expect_tx(&sh.in[warp - 2], in_bytes);
                if (S.load_add)
                    for (int x = 0; x < S.out_bytes / 4096; ++x) tma_load_2d(out + x * 4096, &M.add, &sh.in[warp - 2], col + x * (E.f32 ? 32 : 64), row);
                if (S.load_aux) tma_load_2d(aux, &M.aux, &sh.in[warp - 2], col, row);
            }
            ++asked;
            ahead.next(G, E, unit, set, turn);
        };
        if (ok && !SWAP && TMA) ask();
        // the pass's bias, loaded before its products are there
        float *biases = reinterpret_cast<float*>(&sh) - 4 * S.sets * S.turns * kLinBias / 4 + (warp - 2) * 64, b0 = 0.f, b1 = 0.f;
        auto ask_bias = [&](int64_t j) {
            if (OP != OP_FWD || SWAP || !E.bias) return;
            b0 = j + lane < E.cols ? E.bias[j + lane] : 0.f;
            b1 = j + 32 + lane < E.cols ? E.bias[j + 32 + lane] : 0.f;
        };
        // SUMS: the warp's group g of 32 columns, of four
        auto group_of = [&](int g) { return S.gw == 64 ? 64 * (turn + 2 * (g >> 1)) + 32 * (g & 1) : 32 * (turn + 2 * g); };
        Accumulators A;
        while (ok && way.next(G, unit, s)) {
            const bool sums = takes_sums<OP, SWAP>(E, s);
            int acc = A.next(sums);
            if (S.sets == 2 && acc != set) {
                A.used(acc, sums);
                continue;
            }
            const int64_t i = (int64_t)s.mt * (PAIR ? 256 : 128 * G.sub) + 128 * rank + r, j0 = (int64_t)s.nt * G.bn;
            const int across = (G.bn + S.gw - 1) / S.gw, most = across * parts_of<PAIR>(G, s);  // passes
            float* part = s.slot < 0 ? nullptr : G.part + ((int64_t)s.slot * (PAIR ? 2 : 1) + rank) * 128 * G.bn;
            ask_bias(j0 + turn % across * S.gw);
            // without TMA a warp loads for itself: for its first pass before the products are there
            auto copy_in = [&](int64_t row, int col) {
                if (TMA || SWAP || row >= E.rows || col >= E.cols) return;
                if (S.load_add) slab_copy<true>(out, const_cast<void*>(E.add), E.f32, row, E.rows, col, E.cols, S.gw, E.pitch);
                if (S.load_aux) slab_copy<true>(aux, const_cast<uint16_t*>(E.pre_in), 0, row, E.rows, col, E.cols, S.gw, E.pitch);
                __syncwarp();
            };
            if (!part && turn < most) copy_in(i - lane + 128 * (turn / across), (int)j0 + turn % across * S.gw);
            const uint32_t lanes = (uint32_t)(32 * q) << 16, tm1 = sh.tmem + 256 + lanes;
            uint32_t tm = 0;
            auto filled = [&]() {
                acc = A.next(sums);
                tm = sh.tmem + acc * 256 + lanes;
                ok = mbar_wait(&sh.tfull[acc], A.uses[acc] & 1, &sh.abort, G.wait_ns, G.status, WAIT_EPI_TMEM_FULL);
                tc_fence_after();
                return ok;
            };
            auto emptied = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR)
                        arrive_first(&sh.tempty[acc]);
                    else
                        mbar_arrive(&sh.tempty[acc]);
                }
                A.used(acc, sums);
            };
            // SUMS: db of the tile, as the blocks' sums come: the thread's row's, or (SWAP, where all rows are alike) column `lane`'s of a
            // group of 32 to each warp
            float b = 0.f;
            auto add_db = [&]() {
                if (!SUMS || OP != OP_WGRAD || !sums || (!SWAP && turn != 0) || (SWAP && group_of(q) >= G.bn)) return;
                uint32_t u[32];
                if (SWAP) {
                    uint32_t low = 0;
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
                        tmem_ld16(tm1 + group_of(q) + h, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int o = 8; o; o >>= 1)
#pragma unroll
                            for (int e = 0; e < o; ++e) u[e] = lane & o ? u[e + o] : u[e];
                        if (h == 0) low = u[0];
                    }
                    u[0] = lane & 16 ? u[0] : low;
                } else {
                    tmem_ld16(tm1, u);
                    tmem_ld_wait();
                }
                b += __uint_as_float(u[0]);
            };
            if (SUMS && s.kb1 - s.kb0 > G.seg) {
                // all blocks' sums, the last written back to where the epilogue finds a tile's
                uint64_t v[4][16];
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[g][e] = 0;
                for (int k0 = s.kb0; k0 < s.kb1; k0 += G.seg) {
                    if (!filled()) break;
                    add_db();
                    const bool last = k0 + G.seg >= s.kb1;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int c = group_of(g);
                        if (c >= G.bn) continue;
#pragma unroll
                        for (int h = 0; h < 16; h += 8) {
                            uint32_t u[32];  // the first 16
                            tmem_ld16(tm + c + 2 * h, u);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                v[g][h + e] = add2(v[g][h + e], two(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])));
                            if (!last) continue;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float a, b;
                                apart(v[g][h + e], a, b);
                                u[2 * e] = __float_as_uint(a), u[2 * e + 1] = __float_as_uint(b);
                            }
                            tmem_st16(tm + c + 2 * h, u);
                        }
                    }
                    if (last)
                        tmem_st_wait();
                    else
                        emptied();
                }
                if (!ok) break;
            } else if (!filled()) {
                break;
            } else {
                add_db();
            }
            if (SWAP || part) {
                for (int k = 0;; ++k) {
                    const int c = SUMS ? group_of(k >> 1) + 16 * (k & 1) : 16 * (turn + S.turns * k);
                    if (SUMS ? k == 8 : c >= G.bn) break;
                    if (c >= G.bn) continue;
                    uint32_t u[32];
                    tmem_ld16(tm + c, u);
                    tmem_ld_wait();
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(u[e]);
                    if (part) {
                        // four columns of all 128 rows in turn
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            reinterpret_cast<float4*>(part)[((c + e) >> 2) * 128 + r] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    } else if (i < G.m) {
                        finish_column<OP>(E, j0 + c, (int)i, v);
                    }
                    if (OP == OP_WGRAD && SWAP && !SUMS && sums) {
                        tmem_ld16(tm1 + c, u);
                        tmem_ld_wait();
                        if (r == 0) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int64_t j = j0 + c + e;
                                const float b = __uint_as_float(u[e]);
                                if (part)
                                    G.dpart[(int64_t)s.slot * 256 + c + e] = b;
                                else if (j < G.n)
                                    E.db[j] = E.accumulate ? fmaf(E.scale, b, E.db[j]) : E.scale * b;
                            }
                        }
                    }
                }
            } else {
                for (int pass = turn; pass < most; pass += S.turns, ++done) {
                    const int sub = pass / across, c0 = (pass - sub * across) * S.gw;
                    const int64_t row = i - lane + 128 * sub;
                    const int col = (int)j0 + c0;
                    if (TMA && in_bytes) {
                        ok = mbar_wait(&sh.in[warp - 2], done & 1, &sh.abort, G.wait_ns, G.status, WAIT_EPI_TMEM_FULL);
                        if (!ok) break;
                    } else if (pass != turn) {
                        copy_in(row, col);
                    }
                    if (OP == OP_FWD && E.bias) {
                        biases[lane] = b0, biases[32 + lane] = b1;
                        __syncwarp();
                        ask_bias(j0 + (pass + S.turns) % across * S.gw);
                    }
#pragma unroll 1
                    for (int c = 0; c < S.gw && c0 + c < G.bn; c += 16) {
                        uint32_t u[32];  // the first 16
                        tmem_ld16(tm + sub * G.bn + c0 + c, u);
                        tmem_ld_wait();
                        float v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(u[e]);
                        if (col + c < E.cols) finish_row<OP>(E, S, out, aux, biases, lane, c, v);
                    }
                    const bool pre = OP == OP_FWD && S.aux_bytes;
                    if (TMA) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            const int step = E.f32 ? 32 : 64;
                            for (int x = 0; row < E.rows && x < S.out_bytes / 4096; ++x)
                                if (col + x * step < E.cols) tma_store_2d(&M.out, out + x * 4096, col + x * step, (int)row);
                            if (pre && row < E.rows && col < E.cols) tma_store_2d(&M.aux, aux, col, (int)row);
                            bulk_commit();
                        }
                        ask();
                    } else {
                        __syncwarp();
                        if (row < E.rows) {
                            slab_copy<false>(out, E.out, E.f32, row, E.rows, col, E.cols, S.gw, E.pitch);
                            if (pre) slab_copy<false>(aux, E.pre_out, 0, row, E.rows, col, E.cols, S.gw, E.pitch);
                        }
                        __syncwarp();
                    }
                }
                if (!ok) break;
            }
            if (OP == OP_WGRAD && !SWAP && turn == 0 && sums) {
                if (!SUMS) {
                    uint32_t u[32];
                    tmem_ld16(tm1, u);
                    tmem_ld_wait();
                    b = __uint_as_float(u[0]);
                }
                if (part)
                    G.dpart[(int64_t)s.slot * 256 + 128 * rank + r] = b;
                else if (i < G.m)
                    E.db[i] = E.accumulate ? fmaf(E.scale, b, E.db[i]) : E.scale * b;
            }
            if (OP == OP_WGRAD && SWAP && SUMS && sums) {
                const int c = group_of(q) + lane;
                const int64_t j = j0 + c;
                if (c < G.bn) {
                    if (part)
                        G.dpart[(int64_t)s.slot * 256 + c] = b;
                    else if (j < G.n)
                        E.db[j] = E.accumulate ? fmaf(E.scale, b, E.db[j]) : E.scale * b;
                }
            }
            emptied();
        }
        if (lane == 0) bulk_wait_read();  // shared memory outlives the stores' reads; the stores end with the grid
        if (!SWAP && lane == 0 && *(volatile int*)&sh.abort)  // loads in flight end before the CTA leaves
            for (uint32_t k = done; k < asked; ++k) mbar_wait_timed(&sh.in[warp - 2], k & 1, G.wait_ns);
    }
    __syncwarp();
    // after a wait that gave up: copies and products in flight end before the CTA leaves
    if (*(volatile int*)&sh.abort) {
        if (threadIdx.x == 0) {
            for (int k = 0; k < kLinMostStages; ++k)  // bits: the parity after a stage's last copy
                if (R.issued & (1u << k)) mbar_wait_timed(&sh.full[k], ((R.bits >> k) & 1) ^ 1, G.wait_ns);
        } else if (threadIdx.x == 32 && rank == 0) {
            if (PAIR)
                commit_pair(&sh.drain);
            else
                umma_commit(&sh.drain);
            mbar_wait_timed(&sh.drain, 0, G.wait_ns);
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

// A tile to a cluster of two or four CTAs, which share the blocks of the contracted axis: each leaves its sums in its shared memory, four
// columns of all 128 rows in turn, and of some of the columns adds all CTAs', in their order, and takes the epilogue.  8 x 2048 -> 2048
// takes 6.8 us so, and 7.7 with parts in memory and a second launch (10.6 in clusters of eight);
// 128 x 4096 -> 4096 11.9 and 16.7; 200 x 4096 -> 4096 17.4 and 23.
constexpr int kSplitThreads = 64 + 32 * 8;
constexpr int kMostSplit = 4;
template <int OP, bool SWAP>
__global__ void __launch_bounds__(kSplitThreads, 1) linear_split_kernel(const __grid_constant__ LinMaps M, const __grid_constant__ LinGemm G,
                                                                       const __grid_constant__ LinEpi E) {
    extern __shared__ __align__(1024) uint8_t ring[];
    LinShared& sh = *reinterpret_cast<LinShared*>(ring + kLinSmem - sizeof(LinShared));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = (int)cluster_rank(), C = G.split;
    // the swizzle goes by the address: all CTAs' are alike, and leave alike
    if (smem_u32(ring) & 1023) {
        if (threadIdx.x == 0) atomicCAS(G.status, 0, (int)WAIT_PROBE);
        return;
    }
    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&M.a);
            tma_prefetch_desc(&M.b);
            sh.abort = 0;
            mbar_init(&sh.tfull[0], 1);
            mbar_init(&sh.drain, 1);
        }
        if (lane < kLinMostStages) mbar_init(&sh.full[lane], 1), mbar_init(&sh.empty[lane], 1);
        fence_barrier_init();
        __syncwarp();
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    int mt, nt;
    tile_of(G, blockIdx.x / C, mt, nt);
    const int kb0 = (int)((int64_t)G.nkb * rank / C), kb1 = (int)((int64_t)G.nkb * (rank + 1) / C);
    const int64_t m0 = (int64_t)mt * 128, n0 = (int64_t)nt * G.bn;
    LinRing R;
    if (warp == 0) {
        const bool isb = lane >= 2;
        const int q = isb ? lane - 2 : lane;
        const int na = G.a_mn ? (int)min((int64_t)2, (G.m - m0 + 63) / 64) : 1, nb = G.b_mn ? (int)min((int64_t)(G.bn + 63) / 64, (G.n - n0 + 63) / 64) : 1;
        const uint32_t bytes = (G.a_mn ? na * 8192 : 16384) + (G.b_mn ? nb * 8192 : G.b_box * 128);
        const bool mn = isb ? G.b_mn : G.a_mn, mine = q < (isb ? nb : na);
        const int64_t r0 = isb ? n0 : m0;
        for (int kb = kb0; kb < kb1; ++kb) {
            const bool ok = mbar_wait(&sh.empty[R.stage], R.parity() ^ 1, &sh.abort, G.wait_ns, G.status, WAIT_PRODUCER_EMPTY);
            if (!__all_sync(~0u, ok)) break;
            uint64_t* bar = &sh.full[R.stage];
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (mine) {
                uint8_t* to = ring + R.stage * G.stage_bytes + (isb ? 16384 : 0) + q * 8192;
                if (mn)
                    tma_load_2d(to, isb ? &M.b : &M.a, bar, (int)(r0 + 64 * q), 64 * kb);
                else
                    tma_load_2d(to, isb ? &M.b : &M.a, bar, 64 * kb, (int)r0);
            }
            R.issued |= 1u << R.stage;
            R.next(G.stages);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_bf16(128, G.bn, G.a_mn, G.b_mn);
            const uint32_t astep = G.a_mn ? 2048 : 32, bstep = G.b_mn ? 2048 : 32, alead = G.a_mn ? 8192 : 16, blead = G.b_mn ? 8192 : 16;
            bool ok = true;
            for (int kb = kb0; ok && kb < kb1; ++kb) {
                ok = mbar_wait(&sh.full[R.stage], R.parity(), &sh.abort, G.wait_ns, G.status, WAIT_MMA_FULL);
                if (!ok) break;
                tc_fence_after();
                const uint32_t as = smem_u32(ring + R.stage * G.stage_bytes), bs = as + 16384;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_bf16(sh.tmem, sdesc(as + k * astep, alead, 1024, SWZ_128B), sdesc(bs + k * bstep, blead, 1024, SWZ_128B), idesc, kb > kb0 || k > 0);
                umma_commit(&sh.empty[R.stage]);
                R.next(G.stages);
            }
            if (ok) umma_commit(&sh.tfull[0]);
        }
    } else {
        // all operands are read when the products are done, and their place is the sums'
        const int q = warp & 3, turn = (warp - 2) >> 2;
        if (mbar_wait(&sh.tfull[0], 0, &sh.abort, G.wait_ns, G.status, WAIT_EPI_TMEM_FULL)) {
            tc_fence_after();
            float4* to = reinterpret_cast<float4*>(ring) + 32 * q + lane;
            for (int c = 16 * turn; c < G.bn; c += 32) {
                uint32_t u[32];
                tmem_ld16(sh.tmem + ((uint32_t)(32 * q) << 16) + c, u);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    to[((c + e) >> 2) * 128] = make_float4(__uint_as_float(u[e]), __uint_as_float(u[e + 1]), __uint_as_float(u[e + 2]), __uint_as_float(u[e + 3]));
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    // after a wait that gave up: copies and products in flight end before the CTA leaves
    if (*(volatile int*)&sh.abort) {
        if (threadIdx.x == 0) {
            for (int k = 0; k < kLinMostStages; ++k)
                if (R.issued & (1u << k)) mbar_wait_timed(&sh.full[k], ((R.bits >> k) & 1) ^ 1, G.wait_ns);
        } else if (threadIdx.x == 32) {
            umma_commit(&sh.drain);
            mbar_wait_timed(&sh.drain, 0, G.wait_ns);
        }
    }
    cluster_sync();  // all CTAs' sums are there
    const int quads = G.bn / 4, from = quads * rank / C, to = quads * (rank + 1) / C;
    float4* mine = reinterpret_cast<float4*>(ring) + quads * 128;  // behind the sums: the CTA's own columns, row by row
    if (warp >= 2) {
        for (int f = threadIdx.x - 64; f < (to - from) * 128; f += 256) {
            const int row = f & 127, c4 = from + (f >> 7);
            float4 x[kMostSplit];
#pragma unroll
            for (int k = 0; k < kMostSplit; ++k) {
                if (k >= C) continue;
                const uint32_t at = remote(reinterpret_cast<const float4*>(ring) + c4 * 128 + row, k);
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[k].x), "=f"(x[k].y), "=f"(x[k].z), "=f"(x[k].w) : "r"(at));
            }
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kMostSplit; ++k)
                if (k < C) v[0] += x[k].x, v[1] += x[k].y, v[2] += x[k].z, v[3] += x[k].w;
            if (SWAP)
                finish_column<OP>(E, n0 + 4 * c4, (int)m0 + row, v);
            else  // a row's quads, turned by the row so that both ways are without conflicts
                mine[row * (to - from) + ((f >> 7) + row) % (to - from)] = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (!SWAP) {
            named_bar_sync(2, 256);
            const int wide = to - from;
            const int row = 16 * (warp - 2);
            if (m0 + row < G.m)
                for (int c = lane; c < 4 * wide; c += 32) {
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = reinterpret_cast<const float*>(mine + (row + e) * wide + ((c >> 2) + row + e) % wide)[c & 3];
                    finish_column<OP>(E, m0 + row, (int)n0 + 4 * from + c, v);
                }
        }
    }
    cluster_sync();  // and read
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, 256);
    }
}

// The tiles that were cut, from their parts in order: a block has 32 columns of so many rows that `ways` threads share the parts of
// four values of a row; the sums go through shared memory to rows of 32 columns (SWAP: are columns of rows already).
template <int OP, bool SWAP>
__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ LinGemm G, const __grid_constant__ LinEpi E, int pair, int ways) {
    __shared__ float4 red[256];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int ctas = pair ? 2 : 1, high = 32 / ways;                      // rows of a block
    const int across = (G.bn + 31) / 32, down = ctas * 128 / high;        // blocks of a tile
    const int e = blockIdx.x / (across * down);
    const int64_t u0 = (int64_t)e * G.nkb / G.share, u1 = ((int64_t)(e + 1) * G.nkb - 1) / G.share;
    if (u0 == u1) return;  // this tile was a unit's alone
    int mt, nt;
    tile_of(G, G.whole + e, mt, nt);
    const int block = (int)(blockIdx.x - e * across * down), c0 = block / down * 32, r0 = block % down * high;
    const int way = threadIdx.x / (8 * high), in = threadIdx.x % (8 * high), row = r0 + in % high, quad = in / high;
    const int64_t apart = (int64_t)ctas * 32 * G.bn;
    const float4* p = reinterpret_cast<const float4*>(G.part) + (int64_t)(row >> 7) * 32 * G.bn + (c0 / 4 + quad) * 128 + (row & 127);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c0 + 4 * quad < G.bn) {
#pragma unroll 8
        for (int64_t u = u0 + way; u <= u1; u += ways) {
            const float4 x = __ldcg(p + (2 * u + (u == u0)) * apart);
            s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
        }
    }
    red[threadIdx.x] = s;
    __syncthreads();
    if (SWAP) {
        if (way == 0) {
            for (int w = 1; w < ways; ++w) {
                const float4 x = red[w * 8 * high + in];
                s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
            }
            float v[4] = {s.x, s.y, s.z, s.w};
            if (c0 + 4 * quad < G.bn) finish_column<OP>(E, (int64_t)nt * G.bn + c0 + 4 * quad, mt * 128 + row, v);
        }
    } else {
        const int lane = threadIdx.x & 31;
        // a warp's rows are neighbours: four, or one where the parts are shared
        auto rows = [&](auto count) {
            constexpr int N = decltype(count)::value;
            for (int r = N * (threadIdx.x >> 5); r < high; r += 8 * N) {
                float v[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float* at = reinterpret_cast<const float*>(red + lane / 4 * high + r + e) + (lane & 3);
                    v[e] = 0.f;
                    for (int w = 0; w < ways; ++w) v[e] += at[w * 8 * high * 4];
                }
                const int64_t i = (int64_t)mt * 128 * ctas + r0 + r;
                if (i < G.m && c0 + lane < G.bn) finish_column<OP>(E, i, nt * G.bn + c0 + lane, v);
            }
        };
        if (high == 32)
            rows(std::integral_constant<int, 4>{});
        else
            rows(std::integral_constant<int, 1>{});
    }
    // db of the tile: 256 values, by the tile's first block
    if (OP == OP_WGRAD && E.db && (SWAP ? mt : nt) == 0 && block == 0) {
        float b = 0.f;
        for (int64_t u = u0; u <= u1; ++u) b += __ldcg(G.dpart + (2 * u + (u == u0)) * 256 + threadIdx.x);
        const int64_t j = SWAP ? (int64_t)nt * G.bn + threadIdx.x : (int64_t)mt * 128 * ctas + threadIdx.x;
        const bool there = SWAP ? (int)threadIdx.x < G.bn && j < G.n : (int)threadIdx.x < 128 * ctas && j < G.m;
        if (there) E.db[j] = E.accumulate ? fmaf(E.scale, b, E.db[j]) : E.scale * b;
    }
}

struct LinPlan {
    LinGemm g;
    bool pair, swap;
    bool cut;   // some tile is in parts
    bool sums;  // SUMS
};

// Both launches of a product; instantiated for each direction in a file of its own.
template <int OP>
cf_status launch_linear(const LaunchCtx& ctx, const LinPlan& P, const LinMaps& M, const LinEpi& E);

#ifdef CF_LINEAR_OP
namespace {
template <bool PAIR, bool SWAP, bool TMA, bool SUMS>
cf_status run_linear(const LaunchCtx& ctx, const LinPlan& P, const LinMaps& M, const LinEpi& E) {
    auto kernel = linear_gemm_kernel<PAIR, CF_LINEAR_OP, SWAP, TMA, SUMS>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinSmem) != cudaSuccess) return cudaGetLastError(), CF_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(P.g.units * (PAIR ? 2 : 1)));
    cfg.blockDim = dim3(threads_of_linear(SUMS));
    cfg.dynamicSmemBytes = kLinSmem;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = PAIR ? 2 : 1;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = PAIR ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, M, P.g, E) != cudaSuccess) return cudaGetLastError(), CF_ERR_CUDA;
    if (!P.cut) return CF_OK;
    const int64_t tiles = P.g.rest / P.g.nkb, parts = ((int64_t)P.g.nkb + P.g.share - 1) / P.g.share + 1;
    int ways = 1;
    while (ways < 8 && 4 * ways < parts) ways *= 2;
    cfg.gridDim = dim3((unsigned)(tiles * ((P.g.bn + 31) / 32) * ((PAIR ? 2 : 1) * 4 * ways)));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, linear_join_kernel<CF_LINEAR_OP, SWAP>, P.g, E, PAIR ? 1 : 0, ways) != cudaSuccess)
        return cudaGetLastError(), CF_ERR_CUDA;
    return CF_OK;
}
template <bool SWAP>
cf_status run_split(const LaunchCtx& ctx, const LinPlan& P, const LinMaps& M, const LinEpi& E) {
    auto kernel = linear_split_kernel<CF_LINEAR_OP, SWAP>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinSmem) != cudaSuccess) return cudaGetLastError(), CF_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(P.g.tm * P.g.tn * P.g.split));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = kLinSmem;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)P.g.split;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, M, P.g, E) != cudaSuccess) return cudaGetLastError(), CF_ERR_CUDA;
    return CF_OK;
}
}  // namespace

template <>
cf_status launch_linear<CF_LINEAR_OP>(const LaunchCtx& ctx, const LinPlan& P, const LinMaps& M, const LinEpi& E) {
    if constexpr (CF_LINEAR_OP != OP_WGRAD)
        if (P.g.split) return P.swap ? run_split<true>(ctx, P, M, E) : run_split<false>(ctx, P, M, E);
    auto run = [&](auto sums) {
        constexpr bool kSums = decltype(sums)::value;
        if (P.swap) return run_linear<false, true, true, kSums>(ctx, P, M, E);
        if (P.pair) return P.g.st.tma ? run_linear<true, false, true, kSums>(ctx, P, M, E) : run_linear<true, false, false, kSums>(ctx, P, M, E);
        return P.g.st.tma ? run_linear<false, false, true, kSums>(ctx, P, M, E) : run_linear<false, false, false, kSums>(ctx, P, M, E);
    };
    return P.sums ? run(std::true_type{}) : run(std::false_type{});
}
#endif

}  // namespace cf
