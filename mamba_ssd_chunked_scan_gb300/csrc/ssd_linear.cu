// Matrix product with bias, activation and residual in its epilogue, and its gradients:
//   ssd_linear_tc       D = A B^T over 128 x TN tiles on the tensor cores (tcgen05), the epilogue on
//                       the accumulator as it leaves tensor memory
//   ssd_linear_join     the sum of a split contraction's parts, then the same epilogue
//   ssd_linear_dpre     dy act'(pre) (rounded to bf16, the gradients' operand) and the shares of dbias
//   ssd_linear_dbias    dbias from the shares, in a fixed order
//
// One persistent CTA per SM walks tiles (or tiles' parts along the contraction): one thread loads
// 128-byte-wide operand tiles by TMA into a ring of stages, one issues the MMAs, eight warps run the
// epilogue of the previous tile from the other half of tensor memory meanwhile.  A thread holds one row of 32 columns
// there; blocks of 32 rows x 64 bytes go through shared memory, so that memory sees whole sectors.  Where there are enough
// tiles, two SMs of a cluster share one of 256 rows (PAIR): each holds the accumulator of its 128 rows and loads
// its rows of A and half of B's, and the first one issues the MMAs of both.  Operands come from L2, and a pair asks
// for 64 bytes per SM and cycle of bf16 MMAs where a single CTA asks for 96, more than L2 gives.
// Operands are bf16 or e4m3; a bf16 operand may also be stored with its contraction along the rows
// (dx = dpre W reads W so, dw = dpre^T x both), which the shared-memory descriptors express: no
// operand is ever transposed in memory.
//
// Up to 64 rows of x (decoding) the product is computed transposed, D^T = W x^T: W's rows
// fill the 128 rows of a tile and x is the narrow operand, so the MMAs and the loads are W's
// and almost nothing is padding; its bound is W's one pass from HBM.
//
// Measured: 16384 x 10240 x 2560 bf16 430-435 us back to back (1.97 PFLOP/s; the library's product 419) and 507 under
// the power cap (1.69; the library's sustained rate 1.72); both gradients of it 906-928 us (library 880); e4m3
// 4099 x 2560 x 5120 with its residual 46-49 us, from HBM; 8 rows of e4m3 by 10240 x 2560 8.1 us in a graph, of which
// W's bytes need 3.9, of bf16 12.5 (7.7).  dpre of 8192 x 5120 42 us (6.0 TB/s).
//
// Sums are fp32 in tensor memory.  Tiles run in waves of one per SM (or pair); those of the last wave, which would
// leave SMs idle, are split along the contraction into parts that are summed in a fixed order
// (ssd_linear_join), so results are deterministic.
#include <string.h>

#include <atomic>

#include "ssd_common.cuh"
#include "ssd_kernels.h"
#include "ssd_unpack.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (4 + kEpiWarps);   // warp 0 loads, 1 MMAs, 2 tensor memory, 4-11 epilogue
constexpr int kRowB = 128;             // bytes of the contraction per tile row and stage
constexpr int kTileM = kLinearTileRows;
constexpr uint32_t kWhereEmpty = 61, kWhereFull = 62, kWhereAccFree = 63, kWhereAcc = 64, kWhereDrain = 65;

// TB: columns of the tile whose operand rows this CTA loads (half of them in a pair)
template <int TN, bool PAIR>
struct Cfg {
    static constexpr int TB = PAIR ? TN / 2 : TN;
    static constexpr uint32_t kA = kTileM * kRowB, kB = TB * kRowB, kStage = kA + kB;
    static constexpr int kStages = TB >= 256 ? 4 : TB >= 128 ? 6 : TB >= 64 ? 8 : TB >= 32 ? 9 : 10;
    static constexpr uint32_t kCols = 2 * TN < 32 ? 32 : 2 * TN;   // two accumulators
    static constexpr uint32_t kBlocks = kStages * kStage;                  // the epilogue warps' 32 x 64-byte blocks
    static constexpr uint32_t kVec = kBlocks + kEpiWarps * 2048;           // bias and w_scales of two tiles' columns
    static constexpr size_t kSmem = 1024 + (size_t)kVec + 2 * 2 * TN * 4;
};

struct LinearParams {
    CUtensorMap tm_a, tm_b;
    LinearArgs a;
    int tiles_r, tiles_c;   // tiles over D's rows and columns
    int kblocks;            // 128-byte blocks of the contraction
    int whole;              // tiles [0, whole) are computed whole, the others in `splits` parts
    int splits;
    int items;              // whole + (tiles_r * tiles_c - whole) * splits
    int per;                // blocks per part
};

// What a worker does: a tile and its blocks [k0, k1) of the contraction; part: the part's number among all, or -1.
struct Item {
    int r, c, k0, k1, part;
};

struct Small {
    uint64_t full[10], empty[10], acc[2], acc_free[2], done;
    uint32_t tmem_base;
    int abort, never;
};

__device__ __forceinline__ bool lin_wait(Small& sh, const LinearArgs& a, uint64_t* bar, uint32_t parity, uint32_t where, const int* stop) {
    if (ptx::mbar_wait(bar, parity, stop, a.wait_iters)) return true;
    if (!*(volatile int*)&sh.abort) {
        record_error(a.ws, SSD_ERR_TIMEOUT, where);
        *(volatile int*)&sh.abort = 1;
    }
    return false;
}

// Loads into this CTA's shared memory; in a pair the bytes count on the first CTA's barrier (`bar` is its address).
template <bool PAIR>
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* tm, uint32_t bar, int c0, int c1) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], "
            "[%2];" ::"r"(ptx::smem_u32(dst)),
            "l"(tm), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                ptx::smem_u32(dst)),
            "l"(tm), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
}

template <bool E4M3, bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (!PAIR && !E4M3)
        ptx::mma_ss(d, a, b, idesc, acc);
    else if constexpr (!PAIR)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else if constexpr (!E4M3)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
// Arrival on a barrier when the MMAs issued so far are done; in a pair, on the same barrier of both CTAs.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                ptx::smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        ptx::mma_commit(bar);
}
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t ncols) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(slot)), "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        ptx::tmem_alloc(slot, ncols);
    }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
    else
        ptx::tmem_dealloc(taddr, ncols);
}
// Address of `p` in the pair's first CTA.
__device__ __forceinline__ uint32_t in_first(const void* p) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(ptx::smem_u32(p)));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// One lane of the (whole) warp, the same each time.  The loading and the MMA warp run their loops with all lanes and
// only let this one issue: addresses and descriptors then stay in uniform registers, where the instructions want
// them (from a branch that one lane took, each had to be moved there, about 500 cycles per block of four MMAs).
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}
// The same on a barrier where the cluster's other CTA arrives too.  (An acquire of the wait's own: a fence after it
// held the MMAs up for 1600 cycles per tile.)
__device__ __forceinline__ bool cluster_wait(Small& sh, const LinearArgs& a, uint64_t* bar, uint32_t parity, uint32_t where) {
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t it = 0; it < a.wait_iters; ++it) {
        uint32_t ok;
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
            : "=r"(ok)
            : "r"(ptx::smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((it & 63) == 63 && (*(volatile int*)&sh.abort || ptx::globaltimer() - t0 > ptx::kWaitLimitNs)) break;
    }
    if (!*(volatile int*)&sh.abort) {
        record_error(a.ws, SSD_ERR_TIMEOUT, where);
        *(volatile int*)&sh.abort = 1;
    }
    return false;
}
// A wait by a whole warp, whose lanes go on or give up together.
__device__ __forceinline__ bool warp_wait(Small& sh, const LinearArgs& a, uint64_t* bar, uint32_t parity, uint32_t where, const int* stop) {
    return __all_sync(0xffffffffu, lin_wait(sh, a, bar, parity, where, stop));
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Instruction descriptor of kind::f8f6f4: e4m3 A and B (both K-major), fp32 accumulator.
constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// s(v) = 1 / (1 + exp(-v)) with the special-function unit's exponential and reciprocal
// (relative error of a few 2^-22, far below the rounding of the bf16 results).
__device__ __forceinline__ float sigmoid(float v) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-v * kLog2e));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
constexpr float kGeluC = 0.7978845608028654f, kGeluA = 0.044715f;   // sqrt(2 / pi)

// silu(v) = v s(v);  gelu(v) = v (1 + tanh u) / 2 = v s(2u), u = sqrt(2/pi) (v + 0.044715 v^3)
__device__ __forceinline__ float act_value(float v, int act) {
    if (act == SSD_ACT_SILU) return v * sigmoid(v);
    if (act == SSD_ACT_GELU) return v * sigmoid(2.f * kGeluC * (v + kGeluA * v * v * v));
    return v;
}
// (Beyond a thousand either slope is 0 or 1 to the last bit, and squares of arguments would overflow into 0 times infinity.)
__device__ __forceinline__ float act_slope(float v, int act) {
    v = fabsf(v) > 1000.f ? copysignf(1000.f, v) : v;
    if (act == SSD_ACT_SILU) {
        const float s = sigmoid(v);
        return s * (1.f + v * (1.f - s));
    }
    if (act == SSD_ACT_GELU) {
        const float s = sigmoid(2.f * kGeluC * (v + kGeluA * v * v * v));
        return s + v * s * (1.f - s) * 2.f * kGeluC * (1.f + 3.f * kGeluA * v * v);
    }
    return 1.f;
}

// One element of y from v, its sum with scales and bias: the rounded v for the backward pass, activation, and the
// residual's element, asked for before (y may be the residual, so a load here would wait for the stores of other elements).
__device__ __forceinline__ float residual_at(const LinearArgs& a, size_t at) {
    return a.residual ? __bfloat162float(static_cast<const bf16_t*>(a.residual)[at]) : 0.f;
}
__device__ __forceinline__ void finish(const LinearArgs& a, float v, size_t at, float res) {
    if (a.pre) static_cast<bf16_t*>(a.pre)[at] = __float2bfloat16_rn(v);
    static_cast<bf16_t*>(a.y)[at] = __float2bfloat16_rn(act_value(v, a.act) + res);
}

// 32 rows of 64 bytes through shared memory, by a warp: lane r has row r as four 16-byte words, and they leave as whole
// rows (four lanes each).  The words of a row are permuted so that neither side's accesses share a bank.
__device__ __forceinline__ uint8_t* word_at(uint8_t* block, int row, int word) {
    return block + row * 64 + ((word ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ void put_block(uint8_t* block, const uint4 (&w)[4]) {
    const int lane = threadIdx.x & 31;
    __syncwarp();   // the last block has left
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(word_at(block, lane, k)) = w[k];
    __syncwarp();
}
// The block to memory: row r to base + r * pitch bytes, for r < rows.  `bytes` of each row exist; vec: whole 16-byte
// words, aligned.
__device__ __forceinline__ void send_block(const uint8_t* block, uint8_t* base, size_t pitch, int rows, int bytes, bool vec) {
    const int lane = threadIdx.x & 31;
    uint8_t* const blk = const_cast<uint8_t*>(block);
    if (vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2), word = lane & 3;
            const uint4 v = *reinterpret_cast<const uint4*>(word_at(blk, row, word));
            if (row < rows && 16 * word < bytes) *reinterpret_cast<uint4*>(base + row * pitch + 16 * word) = v;
        }
    } else {
        // one row at a time, a bf16 per lane
#pragma unroll 8
        for (int row = 0; row < 32; ++row)
            if (row < rows && 2 * lane < bytes)
                *reinterpret_cast<uint16_t*>(base + row * pitch + 2 * lane) =
                    *reinterpret_cast<const uint16_t*>(word_at(blk, row, lane >> 3) + 2 * (lane & 7));
    }
}

// 32 columns (one row per lane) of a tile from their sums `w`: D's rows `row` to `row` + 31, columns col on.
// `vec`: this chunk's scales (then bias) by column, in shared memory, TN apart; xs: the row's scale.
// r: the residual's elements, asked for ahead (aligned rows) as they lie in memory, whole rows of 64 bytes by four lanes
// each: asked for by a row per lane they hold up the MMAs' operands (16384 x 10240 x 2560 509 us, so 462).
__device__ __forceinline__ void ask_residual(const LinearArgs& a, uint4 (&r)[4], int64_t row, int col) {
    const int lane = threadIdx.x & 31;
    row += lane >> 2;
    col += 8 * (lane & 3);
    const bf16_t* res = static_cast<const bf16_t*>(a.residual) + (size_t)row * a.n + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = make_uint4(0, 0, 0, 0);
        if (row + 8 * i < a.m && col < a.n) r[i] = __ldcs(reinterpret_cast<const uint4*>(res + (size_t)8 * i * a.n));
    }
}
__device__ __forceinline__ void finish_rows(const LinearArgs& a, const uint32_t (&w)[32], uint4 (&r)[4], int64_t row, int col,
                                            float xs, const float* ws, const float* bias, uint8_t* block) {
    const int lane = threadIdx.x & 31;
    const int rows = a.m - row < 32 ? (int)(a.m - row) : 32, cols = a.n - col < 32 ? a.n - col : 32;
    const size_t at = (size_t)row * a.n + col;
    if (a.residual) {
        const bf16_t* res = static_cast<const bf16_t*>(a.residual);
        __syncwarp();
        if (a.vec) {
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(word_at(block, 8 * i + (lane >> 2), lane & 3)) = r[i];
        } else {   // an element per lane and row, all of them asked for before the first is used
            uint16_t e[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
                e[i] = i < rows && lane < cols ? __ldcs(reinterpret_cast<const unsigned short*>(res + at + (size_t)i * a.n + lane)) : 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) *reinterpret_cast<uint16_t*>(word_at(block, i, lane >> 3) + 2 * (lane & 7)) = e[i];
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = *reinterpret_cast<const uint4*>(word_at(block, lane, k));
    }
    float v[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(w[k]);
    if (a.x_scales) {
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const float4 q = *reinterpret_cast<const float4*>(ws + k);
            v[k] *= xs * q.x;
            v[k + 1] *= xs * q.y;
            v[k + 2] *= xs * q.z;
            v[k + 3] *= xs * q.w;
        }
    }
    if (a.bias) {
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const float4 q = *reinterpret_cast<const float4*>(bias + k);
            v[k] += q.x;
            v[k + 1] += q.y;
            v[k + 2] += q.z;
            v[k + 3] += q.w;
        }
    }
    auto pack = [&](uint4 (&o)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t* q = reinterpret_cast<uint32_t*>(&o[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * k + 2 * e], v[8 * k + 2 * e + 1]);
                q[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
    };
    uint4 o[4];
    if (a.pre) {
        pack(o);
        put_block(block, o);
        send_block(block, static_cast<uint8_t*>(a.pre) + at * 2, (size_t)a.n * 2, rows, cols * 2, a.vec);
    }
    if (a.act != SSD_ACT_NONE) {
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = act_value(v[k], a.act);
    }
    if (a.residual) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(&r[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[8 * k + 2 * e] += __uint_as_float(q[e] << 16);
                v[8 * k + 2 * e + 1] += __uint_as_float(q[e] & 0xFFFF0000u);
            }
        }
    }
    pack(o);
    put_block(block, o);
    send_block(block, static_cast<uint8_t*>(a.y) + at * 2, (size_t)a.n * 2, rows, cols * 2, a.vec);
}

// Tile (r, c) of the t-th tile: bands of kBand row tiles walk the columns together, so that the tiles in
// flight share their operands in L2.
constexpr int kBand = 16;
__device__ __forceinline__ void tile_at(const LinearParams& p, int t, int& r, int& c) {
    const int per = kBand * p.tiles_c;
    const int band = t / per, in = t - band * per;
    const int rows = p.tiles_r - band * kBand < kBand ? p.tiles_r - band * kBand : kBand;
    c = in / rows;
    r = band * kBand + in - c * rows;
}
__device__ __forceinline__ Item item_at(const LinearParams& p, int item) {
    Item i;
    i.part = item < p.whole ? -1 : item - p.whole;
    const int t = i.part < 0 ? item : p.whole + i.part / p.splits;
    tile_at(p, t, i.r, i.c);
    i.k0 = i.part < 0 ? 0 : (i.part % p.splits) * p.per;
    i.k1 = i.part < 0 || i.k0 + p.per > p.kblocks ? p.kblocks : i.k0 + p.per;
    return i;
}

// E4M3: 8-bit operands.  AMN / BMN: the operand's contraction runs along its rows in memory (bf16).
// PAIR: two CTAs per tile of 256 rows.
template <int TN, bool E4M3, bool AMN, bool BMN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) ssd_linear_tc(const __grid_constant__ LinearParams p) {
    using C = Cfg<TN, PAIR>;
    constexpr int kRows = PAIR ? 2 * kTileM : kTileM;   // rows of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ Small sh;
    const LinearArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kElems = E4M3 ? 128 : 64;   // contraction elements per stage
    const int rank = PAIR ? (int)cluster_rank() : 0;
    const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x, workers = PAIR ? gridDim.x >> 1 : gridDim.x;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            ptx::mbar_init(&sh.full[i], 1);
            ptx::mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sh.acc[i], 1);
            ptx::mbar_init(&sh.acc_free[i], PAIR ? 2 * kEpiWarps : kEpiWarps);
        }
        ptx::mbar_init(&sh.done, 1);
        sh.abort = 0;
        sh.never = 0;
        ptx::mbar_fence_init();
        ptx::prefetch_tmap(&p.tm_a);
        ptx::prefetch_tmap(&p.tm_b);
    }
    if (warp == 2) tmem_alloc<PAIR>(&sh.tmem_base, C::kCols);
    ptx::tc_fence_before();
    if (PAIR) cluster_sync();   // both CTAs' barriers are there
    else __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tb = sh.tmem_base;
    // So far nothing was read or written that earlier launches may still be working on: this one may start while they
    // end.  Whoever goes on to global memory waits for them.
    if (warp == 3) {
        pdl_wait();
        if (blockIdx.x == 0 && lane == 0 && a.ws && !a.keep_status) a.ws->status = 0;   // a wait gives up seconds after this
        pdl_trigger();   // the join may start on the threads that this grid leaves free
    } else if (warp == 0) {
        // ---------------------------------------------------------------- loads
        pdl_wait();
        uint32_t it = 0, st = 0, phase = 0;
        bool go = true;
        for (int item = worker; go && item < p.items; item += workers) {
            const Item i = item_at(p, item);
            const int row = i.r * kRows + rank * kTileM, col = i.c * TN + rank * C::TB;
            for (int kb = i.k0; kb < i.k1; ++kb) {
                if (it == a.loads) {   // (an injected stall; else more than there are)
                    go = false;
                    break;
                }
                // A pair's loads count on one barrier: both CTAs have to stop at the same block, so neither gives up for what
                // went wrong in it alone (`never`), only for a stage that neither gets back.
                if (it >= (uint32_t)C::kStages &&
                    !warp_wait(sh, a, &sh.empty[st], phase ^ 1, kWhereEmpty, PAIR ? &sh.never : &sh.abort)) {
                    go = false;
                    break;
                }
                uint8_t* dst = sm + st * C::kStage;
                // a pair's loads all count on the first CTA's barrier, which expects the bytes of both
                const uint32_t bar = PAIR ? in_first(&sh.full[st]) : ptx::smem_u32(&sh.full[st]);
                if (elected()) {
                    if (rank == 0) ptx::mbar_expect_tx(&sh.full[st], PAIR ? 2 * C::kStage : C::kStage);
                    if constexpr (AMN) {
#pragma unroll
                        for (int j = 0; j < kTileM / 64; ++j) tma_load_2d<PAIR>(dst + j * 8192, &p.tm_a, bar, row + 64 * j, kb * kElems);
                    } else {
                        tma_load_2d<PAIR>(dst, &p.tm_a, bar, kb * kElems, row);
                    }
                    if constexpr (BMN) {
#pragma unroll
                        for (int j = 0; j < C::TB / 64; ++j)
                            tma_load_2d<PAIR>(dst + C::kA + j * 8192, &p.tm_b, bar, col + 64 * j, kb * kElems);
                    } else {
                        tma_load_2d<PAIR>(dst + C::kA, &p.tm_b, bar, kb * kElems, col);
                    }
                }
                __syncwarp();
                ++it;
                if (++st == (uint32_t)C::kStages) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        // every load that was issued has landed before the CTA may leave (a pair's count on the first's barriers, and
        // the pair leaves together)
        if (PAIR && rank != 0 && !go && lane == 0) {
            // should this CTA have gone a stage further than the first all the same, no barrier tells when that load lands
            const uint64_t t0 = ptx::globaltimer();
            for (uint32_t k = 0; k < kDefaultWaitIters && ptx::globaltimer() - t0 < 1000000; ++k) {}
        }
        if (rank == 0 && lane == 0)
            for (uint32_t i = 0; i < (uint32_t)C::kStages && i < it; ++i) {
                const uint32_t last = ((it - 1 - i) / C::kStages) * C::kStages + i;
                if (!ptx::mbar_wait(&sh.full[i], (last / C::kStages) & 1, &sh.never, a.wait_iters)) {
                    record_error(a.ws, SSD_ERR_TIMEOUT, kWhereDrain);
                    *(volatile int*)&sh.abort = 1;
                }
            }
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------------------------------------ MMAs (a pair's from its first CTA)
            constexpr uint32_t id = E4M3 ? idesc_e4m3(kRows, TN) : ptx::idesc_bf16(kRows, TN, AMN, BMN);
            // the first stage's descriptors; a stage, and 32 bytes of the contraction (or 16 of its rows), further on
            // is an addition in their address field
            const uint32_t base = ptx::smem_u32(sm);
            const uint64_t da0 = AMN ? ptx::sdesc_sw128(base, 8192, 1024) : ptx::sdesc_sw128(base, 16, 1024);
            const uint64_t db0 = BMN ? ptx::sdesc_sw128(base + C::kA, 8192, 1024) : ptx::sdesc_sw128(base + C::kA, 16, 1024);
            constexpr uint32_t ka = (AMN ? 2048 : 32) >> 4, kb_ = (BMN ? 2048 : 32) >> 4;
            pdl_wait();   // (or the limit of the first wait would count the time of the launches before)
            uint32_t tile = 0, st = 0, phase = 0;
            bool go = true;
            for (int item = worker; go && item < p.items; item += workers, ++tile) {
                const Item i = item_at(p, item);
                const int k0 = i.k0, k1 = i.k1;
                const uint32_t buf = tile & 1, d = tb + buf * TN;
                if (tile >= 2) {
                    const uint32_t parity = ((tile >> 1) - 1) & 1;
                    if (PAIR ? !__all_sync(0xffffffffu, cluster_wait(sh, a, &sh.acc_free[buf], parity, kWhereAccFree))
                             : !warp_wait(sh, a, &sh.acc_free[buf], parity, kWhereAccFree, &sh.abort))
                        break;
                }
                ptx::tc_fence_after();
                for (int kb = k0; kb < k1; ++kb) {
                    if (!warp_wait(sh, a, &sh.full[st], phase, kWhereFull, &sh.abort)) {
                        go = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint64_t da = da0 + st * (C::kStage >> 4), db = db0 + st * (C::kStage >> 4);
                    if (elected()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma<E4M3, PAIR>(d, da + k * ka, db + k * kb_, id, kb > k0 || k > 0);
                        mma_commit<PAIR>(&sh.empty[st]);
                    }
                    __syncwarp();
                    if (++st == (uint32_t)C::kStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
                if (go && elected()) mma_commit<PAIR>(&sh.acc[buf]);   // of a sum that is not whole nothing is written
                __syncwarp();
            }
            if (elected()) mma_commit<PAIR>(&sh.done);
            __syncwarp();
            if (!ptx::mbar_wait(&sh.done, 0, &sh.never, a.wait_iters)) record_error(a.ws, SSD_ERR_TIMEOUT, kWhereDrain);
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3;                 // the warp's quarter of tensor memory's lanes
        const int half = (warp - 4) >> 2;       // and half of the columns (all of them in tiles below 64)
        constexpr int kSpan = TN >= 64 ? TN / 2 : TN;
        constexpr int CW = TN < 32 ? TN : 32;   // columns per read of tensor memory
        constexpr bool kMaySwap = TN <= kLinearSwap;
        pdl_wait();
        static_assert(!kMaySwap || kSpan == CW, "a transposed tile's threads have one read each");
        uint8_t* block = sm + C::kBlocks + (warp - 4) * 2048;
        uint32_t tile = 0;
        for (int item = worker; item < p.items; item += workers, ++tile) {
            const Item i = item_at(p, item);
            const int r = i.r, c = i.c;
            const uint32_t buf = tile & 1;
            const bool whole = i.part < 0 && !a.swap;   // rows of y leave from here
            float* vec = reinterpret_cast<float*>(sm + C::kVec) + buf * 2 * TN;
            if (whole && (a.bias || a.x_scales)) {
                // the columns' scales and bias, once per tile, while its MMAs run; the other tile's are still in use
                for (int k = threadIdx.x - 128; k < TN; k += 32 * kEpiWarps) {
                    const int n = c * TN + k;
                    vec[k] = a.x_scales && n < a.n ? __ldg(a.w_scales + n) : 0.f;
                    vec[TN + k] = a.bias && n < a.n ? __ldg(a.bias + n) : 0.f;
                }
                ptx::named_bar(1, 32 * kEpiWarps);
            }
            const int row0 = r * kRows + rank * kTileM + 32 * q, row = row0 + lane;   // D's row of this thread
            const int nrow = a.swap ? a.n : (int)a.m, ncol = a.swap ? (int)a.m : a.n;
            const bool row_ok = row < nrow;
            // the row's scale and bias (transposed: of the row of w)
            const float rs = a.x_scales && row_ok ? __ldg((a.swap ? a.w_scales : a.x_scales) + row) : 1.f;
            const float rb = a.swap && a.bias && row_ok ? __ldg(a.bias + row) : 0.f;
            // the residual of the first 32 columns comes while the MMAs run, that of the next while these are finished
            const bool ask = whole && a.residual && a.vec;
            uint4 res[4], next[4];
            if (ask) ask_residual(a, res, row0, c * TN + (TN >= 64 ? half * kSpan : 0));
            // transposed: the residual's elements and x's scales of this thread's only columns
            float tr[kMaySwap ? CW : 1], tx[kMaySwap ? CW : 1];
            if (kMaySwap && a.swap) {
                const int col = c * TN + (TN >= 64 ? half * kSpan : 0);
#pragma unroll
                for (int k = 0; k < CW; ++k) {
                    const bool in = row_ok && i.part < 0 && col + k < ncol;
                    tr[k] = in ? residual_at(a, (size_t)(col + k) * a.n + row) : 0.f;
                    tx[k] = in && a.x_scales ? rs * __ldg(a.x_scales + col + k) : 1.f;
                }
            }
            bool ok = true;
            if (lane == 0) ok = lin_wait(sh, a, &sh.acc[buf], (tile >> 1) & 1, kWhereAcc, &sh.abort);
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
            // a wait that runs out stops all of the warps, which share the barrier above
            if (whole && (a.bias || a.x_scales)) ok = !ptx::named_bar_any(2, 32 * kEpiWarps, !ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t d = tb + buf * TN + ((uint32_t)(32 * q) << 16) + (TN >= 64 ? half * kSpan : 0);
            const bool idle = TN < 64 && half;
#pragma unroll 1
            for (int j = 0; j < kSpan; j += CW) {
                __syncwarp();
                uint32_t w[CW];
                if (!idle) {
                    if constexpr (CW == 32) ptx::tmem_load32(d + j, w);
                    else ptx::tmem_load16(d + j, w);
                }
                if (j + CW >= kSpan) {   // the accumulator is in registers: the next tile may have it
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR)
                            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_first(&sh.acc_free[buf]))
                                         : "memory");
                        else
                            ptx::mbar_arrive(&sh.acc_free[buf]);
                    }
                }
                const int col = c * TN + (TN >= 64 ? half * kSpan : 0) + j;
                if (idle || row0 >= nrow || col >= ncol) continue;   // the same for the whole warp
                if (i.part >= 0) {
                    // a part, whole: quads of columns, in each the tile's rows, so that a warp's stores lie together
                    float4* part = reinterpret_cast<float4*>(a.parts) + ((size_t)i.part * (TN / 4) + (col - c * TN) / 4) * kRows + row - r * kRows;
#pragma unroll
                    for (int k = 0; k < CW; k += 4)
                        part[(k / 4) * kRows] = make_float4(__uint_as_float(w[k]), __uint_as_float(w[k + 1]), __uint_as_float(w[k + 2]),
                                                            __uint_as_float(w[k + 3]));
                } else if (kMaySwap && a.swap) {
                    // a lane per column of y: 32 of them lie together in a row
                    if (row_ok) {
#pragma unroll
                        for (int k = 0; k < CW; ++k)
                            if (col + k < ncol) finish(a, __uint_as_float(w[k]) * tx[k] + rb, (size_t)(col + k) * a.n + row, tr[k]);
                    }
                } else if constexpr (CW == 32) {
                    const int k = TN >= 64 ? half * kSpan + j : j;
                    if (ask && j + CW < kSpan) ask_residual(a, next, row0, col + CW);
                    finish_rows(a, w, res, row0, col, rs, vec + k, vec + TN + k, block);
#pragma unroll
                    for (int e = 0; e < 4; ++e) res[e] = next[e];
                }
            }
        }
    }
    ptx::tc_fence_before();
    if (PAIR) cluster_sync();   // neither CTA leaves while the other may still use its memory or barriers
    else __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        tmem_dealloc<PAIR>(tb, C::kCols);
    }
}

// y's elements of the tiles that were computed in parts, the parts added in their order.  A part holds quads of D's columns,
// in each the tile's rows.  A thread takes a quad; a warp 4 rows x 8 quads, 64 bytes together on either side.  (Transposed
// products have y's columns along D's rows: there a thread's four values lie in four rows of y.)
__global__ void __launch_bounds__(256) ssd_linear_join(const __grid_constant__ LinearParams p, int tm, int tn) {
    const LinearArgs& a = p.a;
    const int ctas = tm * tn / 1024;
    const int tile = blockIdx.x / ctas, w = (blockIdx.x - tile * ctas) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    int r, c;
    tile_at(p, p.whole + tile, r, c);
    // transposed: 32 rows of one quad per warp
    const int across = a.swap ? 1 : 8, down = 32 / across, groups = tm / down;
    const int row = (w % groups) * down + lane / across, quad = (w / groups) * across + lane % across;
    const float4* part = reinterpret_cast<const float4*>(a.parts) + ((size_t)tile * p.splits * (tn / 4) + quad) * tm + row;
    const int dr = r * tm + row, dc = c * tn + 4 * quad;
    pdl_trigger();
    const bool some = dr < (a.swap ? a.n : a.m) && dc < (a.swap ? a.m : a.n);
    // Launched while the parts are still being made.  Nothing is read before this, the call's scales, bias and residual
    // neither: that the launch before has seen what earlier ones wrote to them does not make it visible here.
    pdl_wait();
    if (!some) return;
    const int ncol = a.swap ? (int)a.m : a.n;
    const float* along = a.swap ? a.x_scales : a.w_scales;   // scales by D's columns
    const float down_scale = a.x_scales ? __ldg((a.swap ? a.w_scales : a.x_scales) + dr) : 1.f;
    float res[4], scale[4], bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool in = dc + e < ncol;
        scale[e] = in && a.x_scales ? down_scale * __ldg(along + dc + e) : 1.f;
        bias[e] = in && a.bias ? __ldg(a.bias + (a.swap ? dr : dc + e)) : 0.f;
        res[e] = in && (a.swap || !a.vec) ? residual_at(a, a.swap ? (size_t)(dc + e) * a.n + dr : (size_t)dr * a.n + dc + e) : 0.f;
    }
    float v[4];
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        const float4 q = __ldcs(part + (size_t)s * (tn / 4) * tm);
        const float u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = s ? v[e] + u[e] : u[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = v[e] * scale[e] + bias[e];
    if (!a.swap && a.vec) {   // n is a multiple of 8: the four columns exist and are aligned
        const size_t at = (size_t)dr * a.n + dc;
        Raw<bf16_t, 4> o;
        if (a.pre) {
            o.set(v);
            o.store(static_cast<bf16_t*>(a.pre) + at);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_value(v[e], a.act);
        if (a.residual) {
            float t[4];
            o.load(static_cast<const bf16_t*>(a.residual) + at);
            o.get(t);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += t[e];
        }
        o.set(v);
        o.store(static_cast<bf16_t*>(a.y) + at);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (dc + e < ncol) finish(a, v[e], a.swap ? (size_t)(dc + e) * a.n + dr : (size_t)dr * a.n + dc + e, res[e]);
    }
}

// dpre = dy act'(pre), rounded to bf16 into rows of ldp elements, and each row slab's sums over its
// rows (of the unrounded products).  A CTA takes 256 columns of up to kSlabRows rows, a warp every eighth row, a lane eight
// columns: together (V = 8: rows are whole 16-byte words) or 32 apart (V = 1).  Bound by HBM: four rows' loads are in
// flight per warp (8192 x 5120 42 us, 89 % of the copy's rate; with pre in 8 bits 47 us, 66 %).
constexpr int kSlabRows = 128, kSlabCols = 256;
// P: the type of pre (e4m3: times its row's scale; two rows in flight, since decoding takes the registers that more warps run on: all
// gradients of 8192 x 2560 to 5120 293 us, with four 297, with eight 309).  CTAs from x.ctas on unpack x (290 us, 100 x 512 to 512 16.3;
// in a launch of its own 293 and 18.3; these figures are of calls in turns: the products are bound by power, and after other work the
// same call takes up to 320).  Where x comes as 8-bit rows, their scales' factors go into dpre before its rounding, so that the product
// with the codes rounds no operand twice; dx's epilogue takes them out.
// X: whether x does.  What only that takes lies in an argument of its own, so that the others stay in registers (in one kernel for both
// single elements of 32768 x 1001 bf16 took 131 us instead of 78, vectors of 8192 x 5120 49 instead of 46).
template <typename P, int V, bool X>
__global__ void __launch_bounds__(256) ssd_linear_dpre(LinearDpreArgs a, const __grid_constant__ LinearDpreRows x) {
    __shared__ float part[8][kSlabCols];
    constexpr int C = 8 / V, kRowsAhead = sizeof(P) == 1 ? 2 : 4;
    pdl_trigger();
    pdl_wait();
    if (X && blockIdx.x >= x.ctas) {
        unpack_flat<bf16_t>(x.expand, blockIdx.x - x.ctas);
        return;
    }
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const unsigned ncol = (unsigned)(a.n + kSlabCols - 1) / kSlabCols, slab = blockIdx.x / ncol, slab_rows = a.slab_rows;
    const int c0 = (int)(blockIdx.x - slab * ncol) * kSlabCols, n0 = c0 + lane * V;
    const int64_t m0 = (int64_t)slab * slab_rows;
    const int rows = a.m - m0 < slab_rows ? (int)(a.m - m0) : (int)slab_rows;
    const bf16_t* dy = static_cast<const bf16_t*>(a.dy) + (size_t)m0 * a.n + n0;
    const P* pre = a.pre ? static_cast<const P*>(a.pre) + (size_t)m0 * a.n + n0 : nullptr;
    bf16_t* dp = a.dpre ? static_cast<bf16_t*>(a.dpre) + (size_t)m0 * a.ldp + n0 : nullptr;
    float sum[C][V] = {};
    if (X && x.ones)
        for (int k = blockIdx.x * 256 + threadIdx.x; k < x.k; k += x.ctas * 256) x.ones[k] = 1.f;
    for (int k0 = w; k0 < rows; k0 += 8 * kRowsAhead) {
        Raw<bf16_t, V> d[kRowsAhead][C];
        Raw<P, V> q[kRowsAhead][C];
        float scale[sizeof(P) == 1 ? kRowsAhead : 1], factor[X ? kRowsAhead : 1];
        if constexpr (X) {
#pragma unroll
            for (int u = 0; u < kRowsAhead; ++u) {
                const int k = k0 + 8 * u;
                factor[u] = x.x_scales && k < rows ? scale_factor(__ldg(x.x_scales + m0 + k)) : 1.f;
                if (x.inv_factors && k < rows && c0 == 0 && lane == 0) x.inv_factors[m0 + k] = 1.f / factor[u];
            }
        }
        if constexpr (sizeof(P) == 1) {
#pragma unroll
            for (int u = 0; u < kRowsAhead; ++u) scale[u] = k0 + 8 * u < rows ? __ldg(a.pre_scales + m0 + k0 + 8 * u) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + 8 * u;
                d[u][c].zero();
                q[u][c].zero();
                if (k < rows && n0 + 32 * c < a.n) {
                    d[u][c].load(dy + (size_t)k * a.n + 32 * c);
                    if (pre) q[u][c].load(pre + (size_t)k * a.n + 32 * c);
                }
            }
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + 8 * u;
                if (k >= rows || n0 + 32 * c >= a.n) continue;
                float v[V], t[V];
                d[u][c].get(v);
                if (pre) {
                    if constexpr (sizeof(P) == 1) {
                        from_codes(q[u][c], t);
#pragma unroll
                        for (int e = 0; e < V; ++e) t[e] *= scale[u];
                    } else {
                        q[u][c].get(t);
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] *= act_slope(t[e], a.act);
                }
                if (dp) {
                    Raw<bf16_t, V> o;
                    if constexpr (X) {
#pragma unroll
                        for (int e = 0; e < V; ++e) t[e] = v[e] * factor[u];
                        o.set(t);
                    } else {
                        o.set(v);
                    }
                    // read next by the products, so left in L2
                    *reinterpret_cast<typename Raw<bf16_t, V>::W*>(dp + (size_t)k * a.ldp + 32 * c) = o.w;
                }
#pragma unroll
                for (int e = 0; e < V; ++e) sum[c][e] += v[e];
            }
    }
    if (!a.shares) return;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) part[w][lane * V + 32 * c + e] = sum[c][e];
    __syncthreads();
    const int n = c0 + threadIdx.x;
    if (n < a.n) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += part[k][threadIdx.x];
        a.shares[(size_t)slab * a.n + n] = t;
    }
}

// dbias[e] = sum over the slabs' shares: 32 columns per CTA, the shares dealt to its 32
// warps, whose sums are added in warp order.
__global__ void __launch_bounds__(1024) ssd_linear_dbias(const float* shares, int nshares, int n, float* dbias) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    float s = 0.f;
    pdl_trigger();
    pdl_wait();   // launched while the shares are still being summed
    if (e < n)
        for (int k = w; k < nshares; k += 32) s += shares[(size_t)k * n + e];
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && e < n) {
        float t = 0.f;
        for (int k = 0; k < 32; ++k) t += part[k][lane];
        dbias[e] = t;
    }
}

// A (rows, inner) matrix read in boxes of `box_rows` rows x 128 bytes, 128-byte swizzle.
bool encode_2d(CUtensorMap* tm, const void* base, int dtype, int64_t inner, int64_t rows, int64_t ld, int box_rows) {
    const auto enc = tensor_map_encoder();
    if (!enc) return false;
    const int es = dtype == SSD_E4M3 ? 1 : 2;
    cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(ld * es)};
    cuuint32_t box[2] = {(cuuint32_t)(kRowB / es), (cuuint32_t)box_rows};
    cuuint32_t step[2] = {1, 1};
    return enc(tm, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
               dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TN, bool E4M3, bool AMN, bool BMN, bool PAIR>
cudaError_t launch_tile(const LinearParams& p, cudaStream_t st) {
    constexpr size_t smem = Cfg<TN, PAIR>::kSmem;
    const auto kern = ssd_linear_tc<TN, E4M3, AMN, BMN, PAIR>;
    // once per device and kernel: the shared-memory opt-in, and the CTAs (pairs) that run at once
    static std::atomic<int> workers[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = PAIR ? 2 : 1;
    int most = workers[dev].load(std::memory_order_acquire);
    if (most == 0) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
        most = device_sms();
        if (PAIR) {
            cfg.gridDim = dim3(most > 1 ? most / 2 * 2 : 2);
            if ((e = cudaOccupancyMaxActiveClusters(&most, kern, &cfg)) != cudaSuccess) return e;
        }
        if (most < 1) return cudaErrorInvalidConfiguration;
        workers[dev].store(most, std::memory_order_release);
    }
    const int n = p.items < most ? p.items : most;
    cfg.gridDim = dim3(PAIR ? 2 * n : n);
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool E4M3, bool AMN, bool BMN>
cudaError_t launch_kind(const LinearParams& p, const LinearPlan& plan, cudaStream_t st) {
    const int tn = plan.tile_n;
    if (plan.pair) return launch_tile<256, E4M3, AMN, BMN, true>(p, st);
    if (tn == 256) return launch_tile<256, E4M3, AMN, BMN, false>(p, st);
    if (tn == 128) return launch_tile<128, E4M3, AMN, BMN, false>(p, st);
    if constexpr (!AMN && !BMN) {
        if (tn == 32) return launch_tile<32, E4M3, AMN, BMN, false>(p, st);
        if (tn == 16) return launch_tile<16, E4M3, AMN, BMN, false>(p, st);
    }
    return launch_tile<64, E4M3, AMN, BMN, false>(p, st);
}

}  // namespace

// How a product of `rows` x `cols` results over a contraction of `kbytes` bytes runs.  Up to kLinearSwap
// rows it is computed transposed.  Otherwise the tile (128 rows by one CTA and 64 to 256 columns, or 256 by 256 by a pair)
// and the parts of the last wave's tiles minimise a count of cycles.  Measured: a 128-byte block of a tile takes
// 520 cycles by a pair and 541 by a CTA at 256 columns, where the MMAs bound it, but 417 at 128 and 390 at 64 (the
// rows of A are read from shared memory for each MMA however few the columns); a tile's start 600; a
// launch's first loads and last epilogue about 15 a column, and 3000 more for clusters; parts 6300 for the
// join and a cycle per 4000 bytes of them, written and read.  (In bursts, us a block over three waves: a pair 0.324, a CTA 0.371, 0.223
// at 128 columns, 0.216 at 64; two parts of 40 tiles of 128 x 256 over 128 blocks 31.3 us, one 48.2.)  Transposed or not (us, weights
// from HBM, in a graph): 64 rows by 10240 x 2560 bf16 13.8 and 13.8, e4m3 9.5 and 9.3; by 2560 x 5120 11.9 and 14.0, 9.3 and 9.8;
// 128 rows 21.7 and 14.1, 14.9 and 9.7; 13.3 and 14.8, 10.3 and 10.4.
static LinearPlan find_plan(int64_t rows, int64_t cols, int64_t kbytes, bool may_swap) {
    LinearPlan best = {};
    const int64_t kblocks = (kbytes + kRowB - 1) / kRowB;
    const bool swap = may_swap && rows <= kLinearSwap;
    const int64_t dr = swap ? cols : rows, dc = swap ? rows : cols;
    double least = 0;
    const int widths[] = {256, 128, 64, 32, 16};
    for (int pair = 1; pair >= 0; --pair)
        for (int tn : widths) {
            if (pair && (swap || tn < 256)) continue;   // narrower, a CTA's tile takes as long, without the cluster's start
            if (swap ? (tn > kLinearSwap || (tn < dc && tn < kLinearSwap) || (tn > 16 && tn / 2 >= dc)) : tn < 64) continue;
            const int64_t tm = pair ? 2 * kTileM : kTileM;
            const int64_t tiles = ((dr + tm - 1) / tm) * ((dc + tn - 1) / tn), workers = pair ? kLinearSMs / 2 : kLinearSMs;
            const double mma = 2.0 * tn + (pair ? 8 : 29), least_block = 365 + 0.4 * tn;
            const double block = mma > least_block ? mma : least_block;
            const int64_t full = tiles / workers, rest = tiles - full * workers;
            for (int s = 1; s <= kLinearMaxSplits && (s == 1 || rest); ++s) {
                const int64_t per = (kblocks + s - 1) / s;
                if (s > 1 && (per < 4 || (kblocks + per - 1) / per != s)) continue;   // every part has blocks
                double cost = (double)full * (kblocks * block + 600) + 15.0 * tn + (pair ? 3000 : 0);
                cost += (double)((rest * s + workers - 1) / workers) * (per * block + 600);
                if (s > 1) cost += 6300 + (double)rest * s * tm * tn * 8 / 4000;
                if (least == 0 || cost < least) {
                    least = cost;
                    best.tile_n = tn;
                    best.splits = s;
                    best.swap = swap;
                    best.pair = pair != 0;
                    best.whole = s > 1 ? full * workers : tiles;
                    best.parts_bytes = s > 1 ? (size_t)rest * s * tm * tn * 4 : 0;
                }
            }
        }
    return best;
}

// The search takes a microsecond or two, which a decoding step would feel twice (sizing and launching): each
// host thread remembers its last few shapes' plans.
LinearPlan linear_plan(int64_t rows, int64_t cols, int64_t kbytes, bool may_swap) {
    struct Known {
        int64_t rows, cols, kbytes;
        bool may_swap;
        LinearPlan plan;
    };
    static thread_local Known known[64];   // rows 0: empty
    Known& k = known[((uint64_t)rows * 0x9E3779B97F4A7C15ull + (uint64_t)cols * 0xC2B2AE3D27D4EB4Full + (uint64_t)kbytes) >> 32 & 63];
    if (k.rows != rows || k.cols != cols || k.kbytes != kbytes || k.may_swap != may_swap)
        k = Known{rows, cols, kbytes, may_swap, find_plan(rows, cols, kbytes, may_swap)};
    return k.plan;
}

cudaError_t launch_linear(const LinearArgs& args, const LinearPlan& plan, cudaStream_t st) {
    LinearParams p;
    memset(&p, 0, sizeof(p));
    p.a = args;
    LinearArgs& a = p.a;
    if (a.wait_iters == 0) {
        a.wait_iters = kDefaultWaitIters;
        a.loads = ~0u;
    }
    a.swap = plan.swap;
    a.vec = a.n % 8 == 0 && ((uintptr_t)a.y & 15) == 0 && ((uintptr_t)a.residual & 15) == 0 && ((uintptr_t)a.pre & 15) == 0;
    const int64_t dr = a.swap ? a.n : a.m, dc = a.swap ? a.m : a.n;
    const int tn = plan.tile_n, es = a.dtype == SSD_E4M3 ? 1 : 2;
    const int tm = plan.pair ? 2 * kTileM : kTileM, tb = plan.pair ? tn / 2 : tn;
    p.tiles_r = (int)((dr + tm - 1) / tm);
    p.tiles_c = (int)((dc + tn - 1) / tn);
    p.kblocks = (int)((a.k * es + kRowB - 1) / kRowB);
    p.splits = plan.splits;
    p.per = (p.kblocks + p.splits - 1) / p.splits;
    p.whole = (int)plan.whole;
    p.items = p.whole + (p.tiles_r * p.tiles_c - p.whole) * p.splits;
    // the wide operand gives D's rows, 128 at a time; operands with their contraction along the rows
    // are read in boxes of 64 x 64
    const LinearOperand& oa = a.swap ? a.w : a.x;
    const LinearOperand& ob = a.swap ? a.x : a.w;
    const bool ea = oa.along_rows ? encode_2d(&p.tm_a, oa.p, a.dtype, dr, a.k, oa.ld, 64)
                                  : encode_2d(&p.tm_a, oa.p, a.dtype, a.k, dr, oa.ld, kTileM);
    const bool eb = ob.along_rows ? encode_2d(&p.tm_b, ob.p, a.dtype, dc, a.k, ob.ld, 64)
                                  : encode_2d(&p.tm_b, ob.p, a.dtype, a.k, dc, ob.ld, tb);
    if (!ea || !eb) return cudaErrorInvalidValue;
    cudaError_t e;
    if (a.dtype == SSD_E4M3) e = launch_kind<true, false, false>(p, plan, st);
    else if (oa.along_rows) e = launch_kind<false, true, true>(p, plan, st);
    else if (ob.along_rows) e = launch_kind<false, false, true>(p, plan, st);
    else e = launch_kind<false, false, false>(p, plan, st);
    if (e != cudaSuccess || p.splits == 1) return e;
    const int rest = p.tiles_r * p.tiles_c - p.whole;
    return launch_kernel(ssd_linear_join, (unsigned)(rest * (tm * tn / 1024)), 256, 0, st, true, p, tm, tn);
}

// Rows of a slab: kSlabRows, which keeps the shares few, or fewer where that would leave SMs idle (both gradients of
// 2307 x 1783 x 656 57 us with 128 rows, 46 with 32).
static int dpre_slab_rows(int64_t m, int n) {
    const int64_t ncol = (n + kSlabCols - 1) / kSlabCols;
    int rows = kSlabRows;
    while (rows > 32 && (m + rows - 1) / rows * ncol < 4 * kLinearSMs) rows /= 2;
    return rows;
}

int64_t linear_dpre_slabs(int64_t m, int n) {
    const int rows = dpre_slab_rows(m, n);
    return (m + rows - 1) / rows;
}

cudaError_t launch_linear_dpre(const LinearDpreArgs& args, const LinearDpreRows& rows, cudaStream_t st) {
    LinearDpreArgs a = args;
    LinearDpreRows x = rows;
    a.slab_rows = dpre_slab_rows(a.m, a.n);
    const int64_t slabs = linear_dpre_slabs(a.m, a.n);
    x.ctas = (unsigned)(slabs * ((a.n + kSlabCols - 1) / kSlabCols));
    const unsigned grid = x.ctas + (x.expand.out ? unpack_flat_ctas(x.expand) : 0);
    const bool codes = a.pre_scales != nullptr;
    const bool vec = a.n % 8 == 0 && ((uintptr_t)a.pre & (codes ? 7 : 15)) == 0;
    const bool from_rows = x.x_scales || x.expand.out;
    auto kern = codes ? (vec ? (from_rows ? ssd_linear_dpre<e4m3_t, 8, true> : ssd_linear_dpre<e4m3_t, 8, false>)
                             : (from_rows ? ssd_linear_dpre<e4m3_t, 1, true> : ssd_linear_dpre<e4m3_t, 1, false>))
                      : (vec ? (from_rows ? ssd_linear_dpre<bf16_t, 8, true> : ssd_linear_dpre<bf16_t, 8, false>)
                             : (from_rows ? ssd_linear_dpre<bf16_t, 1, true> : ssd_linear_dpre<bf16_t, 1, false>));
    const cudaError_t e = launch_kernel(kern, grid, 256, 0, st, true, a, x);
    if (e != cudaSuccess || !a.dbias) return e;
    return launch_kernel(ssd_linear_dbias, (unsigned)((a.n + 31) / 32), 1024, 0, st, true, (const float*)a.shares, (int)slabs, a.n,
                         a.dbias);
}

}  // namespace ssd
