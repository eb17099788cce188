// Gated linear recurrence, one decay per channel and token:
//   ssd_gate_scan_kernel<fwd>  h_t = a_t h_{t-1} + (1 - a_t) x_t,  a_t = 1 / (1 + exp(-g_t)),  y = h
//   ssd_gate_scan_kernel<bwd>  lam_t = dy_t + a_{t+1} lam_{t+1};  dx = (1 - a) lam,
//                              dg = lam (h_{t-1} - x) a (1 - a),  dinit = a_1 lam_1
//   ssd_gate_scan_clear        the workspace's words to zero, which the other two start from
//   ssd_gate_scan_step_kernel  one token from a resident state
//
// Each step is an affine map of the state, and the maps of consecutive steps
// compose: (A2, B2) o (A1, B1) = (A2 A1, A2 B1 + B2).  The work is cut into tiles of
// kMain segments of SEG tokens x kCh channels.  One CTA per SM has sixteen main warps, one per segment, a
// thread holding two channels; three hand-over warps; and a loading warp:
//   loading    takes the next tile by ticket and brings its inputs into a ring of shared-memory stages (TMA), and
//              sends a finished tile's outputs off from the same stage.  Where rows are not aligned to 16 bytes
//              they come by their alignment's classes, and the main warps store the outputs themselves;
//   main       forms the next tile's decays and its segment's map, keeping exp(-g) in registers; then waits for
//              the state that enters its segment of the tile before, walks that segment again and writes the
//              outputs.  So a tile's state has a whole tile's time to arrive;
//   hand-over  one warp composes the segments' maps to the tile's and publishes it; two (a thread per channel) work out the
//              state that enters the tile and from it those that enter the segments.  (With one set of warps for both, a
//              tile's map waited behind the tile before still waiting for its state.)
// Every input is read from HBM once.  The state that enters a tile follows from the maps of the tiles
// before it in its block of kScanBlock tiles and from the state that enters the block, which the last tile
// of the block before publishes: one hand-over per block is a chain, and the order
// in which maps are composed is fixed, so results do not depend on which tile ran first.  A map
// is one 64-bit word per channel that is never zero once written, so the word is its own flag.  Tickets run
// in the order of the sequences: a tile only waits for tiles of smaller tickets, and a CTA works on its own in
// their order, so the smallest unfinished ticket never waits; every wait is bounded all the same.
//
// The backward pass walks the same maps from the end: mu_t = a_t lam_t obeys
// mu_t = a_t (dy_t + mu_{t+1}).  h_{t-1} inside a segment is recomputed from
// the h before it, which is read from y (rounded to y's type once, at every
// SEG-th token); keeping every h would cost as many bytes again as g.
//
// A document's first token cuts the map (A = 0) and takes the document's own state.
//
// Measured: 65536 x 2048 bf16 in one row, strided, 143 us (5.6 TB/s; the bytes need 119 us at the rate of a copy), bound by
// the main warps' two visits and by reads of 5.4 TB/s without the rest; fp32
// 251 us (95 %); 8 x 2048 x 5120 bf16 backward 135 us (6.2 TB/s); 32767 x 1533, 37 documents, 89 us (1536 columns 71):
// elements off alignment are read from shared memory and stored one by one, and tiles are half as long.  (Loaded by
// elements into registers, a tile ahead: 99 us, 65536 x 2047 231 instead of 185, 8 x 2048 x 5119 backward 224 instead of 190.)
//
// a = 1 / (1 + e) and 1 - a = e a are each formed from e = exp(-g), never one from the other: a channel with a long memory
// needs all digits of 1 - a, a gate that closes all digits of a (the initial states' gradient is a_1 lam_1, and what a large
// state leaves behind is a h).  So e is kept between the visits, and the second one takes the reciprocal of 1 + e again.  (With
// a from a kept 1 - a 65536 x 2048 bf16 took 138 us, fp32 250, and a of a gate at -17 was all rounding.)
// Arithmetic on a thread's two channels is packed (f32x2), which rounds each as the scalar form does.
#include <string.h>

#include <atomic>
#include <type_traits>

#include "ssd_common.cuh"
#include "ssd_kernels.h"
#include "ssd_vec.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

constexpr int kMain = kScanSegs;       // main warps: segments per tile
constexpr int kCh = kScanCh;           // channels per tile: two per main or publishing thread, one per thread that takes states
constexpr int kThreads = 32 * (kMain + 2 + 1 + 1);
constexpr int kBlock = kScanBlock;
static_assert(kCh == 64, "two channels per lane, two hand-over warps");

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kWhereTile = 51, kWhereBlock = 52, kWhereStage = 53, kWhereMaps = 54, kWhereState = 55, kWhereDone = 56;

typedef uint64_t f2;   // two floats, one per channel of a thread
__device__ __forceinline__ f2 pk(float a, float b) { return ptx::f2_pack(a, b); }
__device__ __forceinline__ float2 un(f2 v) {
    float2 r;
    ptx::f2_unpack(v, r.x, r.y);
    return r;
}
__device__ __forceinline__ f2 mul(f2 a, f2 b) { return ptx::f2_mul(a, b); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) { return ptx::f2_fma(a, b, c); }
__device__ __forceinline__ f2 add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// a = 1 / (1 + e), m = 1 - a = e a with e = exp(-g) = 2^(-g log2 e), the exponent capped where e would overflow (a is
// then 1e-38, m one).  Power and reciprocal are the special-function unit's, of relative errors up to 2^-22 and 2^-23; the
// exponent's rounding adds |g| 2^-24.  (expf and a rounded reciprocal for fp32 operands cost 65536 x 2048 16 of 272 us
// and left the same error against 64 bits, 1.4e-7.)
__device__ __forceinline__ f2 forget2(f2 g) {   // e
    const float2 t = un(mul(g, pk(-kLog2e, -kLog2e)));
    float e0, e1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(min_nan(t.x, 126.f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(min_nan(t.y, 126.f)));
    return pk(e0, e1);
}
__device__ __forceinline__ f2 decay2(f2 e) {    // a
    const float2 d = un(add(e, pk(1.f, 1.f)));
    float a0, a1;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a0) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a1) : "f"(d.y));
    return pk(a0, a1);
}

template <typename T> struct PairWord;
template <> struct PairWord<bf16_t> { typedef uint32_t type; };
template <> struct PairWord<float> { typedef uint64_t type; };

// Shapes of a kernel instance.  ROWS: rows are not 16-byte aligned.  Those P apart are off alignment by the same
// bytes, so each of P classes is a matrix of its own, of 16-byte aligned rows that start up to P - 1 elements early: a tile
// comes as P boxes, kCh + P columns wide, and a row's elements lie off by its class's shift.
template <typename T, bool ROWS, bool BWD>
struct Shape {
    static constexpr int ES = sizeof(T), P = 16 / ES;
    static constexpr int SEG = scan_seg(BWD, ES == 2 ? SSD_BF16 : SSD_F32, ROWS), TOK = SEG * kMain;
    static constexpr int PITCH = (kCh + (ROWS ? P : 0)) * ES, ARR = TOK * PITCH;   // one operand's tile
    static constexpr int NA = BWD ? 3 : 2;                      // g, x (and dy)
    static constexpr int STAGE = NA * ARR + (BWD ? kMain * PITCH : 0);   // and, backwards, the h before each segment
    static constexpr int NS = 4 * STAGE <= 212 * 1024 ? 4 : 3;
    static constexpr size_t kSmem = 128 + (size_t)NS * STAGE;
    static_assert(!ROWS || (SEG % P == 0 && (!BWD || SEG == P)), "a segment's classes are those of its first P tokens");
};

// The operands' tensor maps: one each, or (ROWS) one a class.
template <typename T, bool ROWS, bool BWD>
struct ScanParams {
    CUtensorMap g, x, y, dy, dg, dx;
    GateScanArgs a;
};
template <typename T>
struct ScanParams<T, true, false> {
    CUtensorMap g[16 / sizeof(T)], x[16 / sizeof(T)];
    GateScanArgs a;
};
template <typename T>
struct ScanParams<T, true, true> {
    CUtensorMap g[16 / sizeof(T)], x[16 / sizeof(T)], dy[16 / sizeof(T)], y[16 / sizeof(T)];
    GateScanArgs a;
};

struct alignas(16) Tile {
    int row, group;        // batch row, channel group
    int step;              // place in the walk of its sequence
    int ntok;              // its tokens; 0: no tile is left
    int64_t t0;            // its first token
    // elements from the start of g, of x, and of a contiguous operand to the tile's first
    int64_t og, ox, oy;
};

template <bool REV, int TOK>
__device__ __forceinline__ Tile tile_of(const GateScanArgs& a, uint32_t k) {
    Tile t;
    const uint32_t per = (uint32_t)(a.batch * a.ngroups);
    const uint32_t c = k / per, r = k - c * per;
    t.row = (int)(r / (uint32_t)a.ngroups);
    t.group = (int)(r - (uint32_t)t.row * a.ngroups);
    t.step = (int)c;
    t.t0 = (REV ? a.nchunks - 1 - c : c) * TOK;
    t.ntok = k < a.ntiles ? (int)(a.seqlen - t.t0 < TOK ? a.seqlen - t.t0 : TOK) : 0;
    const int64_t tok = (int64_t)t.row * a.seqlen + t.t0;
    t.og = tok * a.g_stride + t.group * kCh;
    t.ox = tok * a.x_stride + t.group * kCh;
    t.oy = tok * a.width + t.group * kCh;
    return t;
}

// A document's state rows (the group's channels) on their way to L2 when its tile is found, a tile or more before they are
// needed: a segment that fetches one from HBM holds up its tile, and the tiles behind it, for a microsecond.
__device__ __forceinline__ void expect_state(const float* p, const GateScanArgs& a, int64_t row, int group) {
    if (!p || row < 0) return;
    p += row * a.width + group * kCh;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
    if (group * kCh + 32 < a.width) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + 32));
}

// Documents that start inside a tile, or at the token after it: doc[k] = the
// document that starts at token t0 + k, or -1.  One warp; offsets outside the tile are skipped,
// so nothing they hold can index out of bounds.  Tiles come in the order of the sequence: the 32 offsets about
// where the last tile's were found (`near`) mostly hold all that this one needs, in one load.  Returns the next `near`.
template <int TOK, bool REV>
__device__ int find_docs(const GateScanArgs& a, int64_t t0, int group, int near, int* doc) {
    const int lane = threadIdx.x & 31;
    auto found = [&](int64_t k, int d) {
        doc[k] = d;
        expect_state(a.init, a, d, group);
        if (REV) expect_state(a.enter, a, d - 1, group);   // what enters at the end of the document before
    };
    for (int k = lane; k <= TOK; k += 32) doc[k] = -1;
    int lo = near - (REV ? 24 : 4);
    if (lo < 0) lo = 0;
    constexpr int64_t kNone = (int64_t)1 << 40;
    int64_t k = lo + lane < a.ndocs ? (int64_t)__ldg(a.cu + lo + lane) - t0 : kNone;
    const bool from = lo == 0 || __shfl_sync(0xffffffffu, k, 0) < 0, to = __shfl_sync(0xffffffffu, k, 31) > TOK;
    __syncwarp();
    if (from && to) {
        if (k >= 0 && k <= TOK) found(k, lo + lane);
        return lo + __popc(__ballot_sync(0xffffffffu, k < 0));
    }
    // the first document whose offset is >= t0, 32 probes at a time
    lo = 0;
    int hi = a.ndocs;
    while (lo < hi) {
        const int gap = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * gap - 1;
        const bool below = at < hi && __ldg(a.cu + at) < t0;
        const int n = __popc(__ballot_sync(0xffffffffu, below));
        lo += n * gap;
        if (lo > hi) lo = hi;
        if (lo + gap - 1 < hi) hi = lo + gap - 1;
    }
    for (int d = lo; d < a.ndocs; d += 32) {
        k = d + lane < a.ndocs ? (int64_t)__ldg(a.cu + d + lane) - t0 : kNone;
        if (k >= 0 && k <= TOK) found(k, d + lane);
        if (__all_sync(0xffffffffu, k > TOK)) break;
    }
    return lo;
}

constexpr int kRing = 8;   // tiles whose numbers and documents are kept: more than one above the stages
template <int TOK, bool DOCS>
struct Shared {
    float2 seg[2][kMain][kCh];       // each segment's map per channel (A, B); then .x: the state that enters it
    Tile tile[kRing];
    int doc[DOCS ? kRing : 1][DOCS ? TOK + 1 : 1];
    uint64_t full[4], done[4];       // per stage: inputs there; outputs written
    uint64_t maps[2], told[2], states[2];   // of tiles in turn: the segments' maps are in seg; the tile's is published;
                                            // the states that enter the segments are in seg
    int abort, never;
};

template <typename S>
__device__ __forceinline__ bool bar_wait(S& sh, const GateScanArgs& a, uint64_t* bar, uint32_t parity, uint32_t where) {
    if (ptx::mbar_wait(bar, parity, &sh.abort, a.wait_iters)) return true;
    if (!*(volatile int*)&sh.abort) {
        record_error(a.ws, SSD_ERR_TIMEOUT, where);
        *(volatile int*)&sh.abort = 1;
    }
    return false;
}

// Words that tiles leave for each other: written once per call, zero before.
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void leave(uint64_t* p, uint64_t v) {
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
// A map (A, B): A >= 0 (or NaN) goes out with its sign bit set, so the word is not zero.
__device__ __forceinline__ uint64_t map_word(float A, float B) {
    return ((uint64_t)__float_as_uint(B) << 32) | (__float_as_uint(A) | 0x80000000u);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tm, uint64_t* bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            ptx::smem_u32(dst)),
        "l"(tm), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* tm, uint64_t* bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            ptx::smem_u32(dst)),
        "l"(tm), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* tm, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tm),
                 "r"(ptx::smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
// ---------------------------------------------------------------------- loading warp
template <typename T, bool ROWS, bool DOCS, bool BWD>
__device__ __forceinline__ void loading(const ScanParams<T, ROWS, BWD>& p, uint8_t* sm, Shared<Shape<T, ROWS, BWD>::TOK, DOCS>& sh) {
    typedef Shape<T, ROWS, BWD> H;
    const GateScanArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    auto send = [&](int j) {   // lane 0: tile j's outputs from its stage
        if constexpr (!ROWS) {
            const Tile& t = sh.tile[j % kRing];
            const uint8_t* st = sm + (j % H::NS) * H::STAGE;
            if (BWD) {
                tma_store_3d(&p.dg, st, t.group * kCh, (int)t.t0, t.row);
                tma_store_3d(&p.dx, st + H::ARR, t.group * kCh, (int)t.t0, t.row);
            } else {
                tma_store_3d(&p.y, st + H::ARR, t.group * kCh, (int)t.t0, t.row);
            }
            ptx::bulk_commit();
        }
    };
    int near = 0;            // documents that start before the last tile, about
    int n = 0, filled = 0;   // tiles, and phases of the stages' `full` begun (the end's among them)
    bool go = true;
    for (;; ++n) {
        uint32_t k = 0;
        if (lane == 0) k = a.nchunks > 1 ? atomicAdd(a.ticket, 1u) : (uint32_t)(blockIdx.x + gridDim.x * n);
        k = __shfl_sync(0xffffffffu, k, 0);
        const Tile t = tile_of<BWD, H::TOK>(a, k);
        // the slot's last tile, n - kRing, is done with: a later one's outputs have been waited for
        if (lane == 0) sh.tile[n % kRing] = t;
        if (DOCS && t.ntok) near = find_docs<H::TOK, BWD>(a, t.t0, t.group, near, sh.doc[n % kRing]);
        const int st = n % H::NS;
        if (n >= H::NS) {
            if (lane == 0) {
                go = bar_wait(sh, a, &sh.done[st], ((n / H::NS) - 1) & 1, kWhereDone);
                if (go) send(n - H::NS);
                ptx::bulk_wait_read0();
            }
            go = __shfl_sync(0xffffffffu, (int)go, 0) != 0;
            if (!go) break;
        }
        if (n == a.loads) break;   // (an injected stall; else negative)
        __syncwarp();
        uint64_t* full = &sh.full[st];
        ++filled;
        if (lane == 0) {
            if (!t.ntok) {
                ptx::mbar_arrive(full);
            } else {
                ptx::mbar_expect_tx(full, H::STAGE);
                if constexpr (!ROWS) {
                    uint8_t* dst = sm + st * H::STAGE;
                    const int c = t.group * kCh, t0 = (int)t.t0;
                    tma_load_3d(dst, &p.g, full, c, t0, t.row);
                    tma_load_3d(dst + H::ARR, &p.x, full, c, t0, t.row);
                    if (BWD) {
                        tma_load_3d(dst + 2 * H::ARR, &p.dy, full, c, t0, t.row);
                        // the h before each segment: every SEG-th row from t0 - 1 (before the sequence: zeros)
                        tma_load_3d(dst + H::NA * H::ARR, &p.y, full, c, t0 - 1, t.row);
                    }
                }
            }
        }
        if (!t.ntok) break;
        if constexpr (ROWS) {
            // lane j: the tile's tokens j, j + P, ...; lane P, backwards: the h before each segment
            __syncwarp();
            uint8_t* dst = sm + st * H::STAGE;
            const int c = t.group * kCh;
            const int64_t r = (int64_t)t.row * a.seqlen + t.t0 + (lane < H::P ? lane : -1);
            const int k = (int)(r & (H::P - 1)), q = (int)(r >> (H::P == 8 ? 3 : 2));
            if (lane < H::P) {
                dst += lane * (H::ARR / H::P);
                tma_load_2d(dst, &p.g[k], full, c, q);
                tma_load_2d(dst + H::ARR, &p.x[k], full, c, q);
                if constexpr (BWD) tma_load_2d(dst + 2 * H::ARR, &p.dy[k], full, c, q);
            }
            if constexpr (BWD)
                if (lane == H::P) tma_load_2d(dst + H::NA * H::ARR, &p.y[k], full, c, q);
        }
    }
    if (lane != 0) return;
    // the outputs of the tiles still in stages, then everything in flight
    for (int j = n - H::NS + 1 > 0 ? n - H::NS + 1 : 0; go && j < n; ++j) {
        go = bar_wait(sh, a, &sh.done[j % H::NS], (j / H::NS) & 1, kWhereDone);
        if (go) send(j);
    }
    for (int st = 0; st < H::NS && st < filled; ++st) {
        const int last = ((filled - 1 - st) / H::NS) * H::NS + st;
        if (!ptx::mbar_wait(&sh.full[st], (last / H::NS) & 1, &sh.never, a.wait_iters)) record_error(a.ws, SSD_ERR_TIMEOUT, kWhereStage);
    }
    ptx::bulk_wait0();
}

// ---------------------------------------------------------------------- hand-over warps
template <bool REV, typename S>
__device__ __forceinline__ void publish_maps(const GateScanArgs& a, S& sh) {
    const int lane = threadIdx.x & 31;   // channels 2 * lane, 2 * lane + 1
    for (int n = 0;; ++n) {
        if (!bar_wait(sh, a, &sh.maps[n & 1], (n >> 1) & 1, kWhereMaps)) return;
        const Tile t = sh.tile[n % kRing];
        if (!t.ntok) return;
        if (t.step % kBlock != kBlock - 1 && t.step != a.nchunks - 1 && !a.mute) {   // another tile of the block needs it
            float4 q[kMain];
#pragma unroll
            for (int k = 0; k < kMain; ++k) q[k] = *reinterpret_cast<const float4*>(&sh.seg[n & 1][REV ? kMain - 1 - k : k][2 * lane]);
            float A0 = 1.f, B0 = 0.f, A1 = 1.f, B1 = 0.f;
#pragma unroll
            for (int k = 0; k < kMain; ++k) {
                B0 = fmaf(q[k].x, B0, q[k].y);
                B1 = fmaf(q[k].z, B1, q[k].w);
                A0 *= q[k].x;
                A1 *= q[k].z;
            }
            uint64_t* to = a.maps + (((int64_t)t.row * a.ngroups + t.group) * a.nchunks + t.step) * kCh + 2 * lane;
            leave(to, map_word(A0, B0));
            leave(to + 1, map_word(A1, B1));
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.told[n & 1]);
    }
}
template <bool REV, typename S>
__device__ __forceinline__ void take_states(const GateScanArgs& a, S& sh) {
    const int c = threadIdx.x - 32 * kMain, lane = threadIdx.x & 31;   // channel of the tile
    for (int n = 0;; ++n) {
        if (!bar_wait(sh, a, &sh.maps[n & 1], (n >> 1) & 1, kWhereMaps)) return;
        const Tile t = sh.tile[n % kRing];
        float2 (*seg)[kCh] = sh.seg[n & 1];
        if (!t.ntok) return;
        const int ch = t.group * kCh + c;
        const int in_block = t.step % kBlock, block = t.step / kBlock;
        const bool more = t.step != a.nchunks - 1, closes = in_block == kBlock - 1;
        const int64_t line = (int64_t)t.row * a.ngroups + t.group;
        uint64_t* maps = a.maps + (line * a.nchunks + (int64_t)block * kBlock) * kCh + c;
        uint64_t* carry = a.carry + (line * a.nblocks + block) * kCh + c;
        // the predecessors' maps and the block's state: all that are missing are asked for at once, so a
        // round takes one trip to L2 however many there are
        uint64_t w[kBlock - 1], cw = 1;
#pragma unroll
        for (int p = 0; p < kBlock - 1; ++p) w[p] = p < in_block ? peek(maps + p * kCh) : 1;
        if (block > 0) cw = peek(carry - kCh);
        uint64_t since = 0;
        for (uint32_t it = 1;; ++it) {
            bool missing = cw == 0;
#pragma unroll
            for (int p = 0; p < kBlock - 1; ++p) missing = missing || w[p] == 0;
            if (!missing) break;
            if (it == 1) since = ptx::globaltimer();
            if ((it & 15) == 0 && (it > a.wait_iters || *(volatile int*)&sh.abort || ptx::globaltimer() - since > kWaitNs)) {
                record_error(a.ws, SSD_ERR_TIMEOUT, cw == 0 ? kWhereBlock : kWhereTile);
                *(volatile int*)&sh.abort = 1;
                break;
            }
#pragma unroll
            for (int p = 0; p < kBlock - 1; ++p)
                if (w[p] == 0) w[p] = peek(maps + p * kCh);
            if (cw == 0) cw = peek(carry - kCh);
        }
        float h = 0.f;
        if (block > 0) h = __uint_as_float((uint32_t)(cw >> 32));
        else if (!a.cu && a.enter && ch < a.width) h = __ldg(a.enter + (int64_t)t.row * a.width + ch);
#pragma unroll
        for (int p = 0; p < kBlock - 1; ++p)
            if (p < in_block) h = fmaf(__uint_as_float((uint32_t)w[p] & 0x7FFFFFFFu), h, __uint_as_float((uint32_t)(w[p] >> 32)));
        float2 m[kMain];
#pragma unroll
        for (int k = 0; k < kMain; ++k) m[k] = seg[REV ? kMain - 1 - k : k][c];
        if (!bar_wait(sh, a, &sh.told[n & 1], (n >> 1) & 1, kWhereMaps)) return;   // the maps have been read
#pragma unroll
        for (int k = 0; k < kMain; ++k) {
            seg[REV ? kMain - 1 - k : k][c].x = h;
            h = fmaf(m[k].x, h, m[k].y);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.states[n & 1]);
        if (more && closes) leave(carry, ((uint64_t)__float_as_uint(h) << 32) | 1u);
        // the state that leaves the sequence: the final state, or the initial state's gradient
        if (!more && !a.cu && a.leave && ch < a.width) a.leave[(int64_t)t.row * a.width + ch] = h;
    }
}

// ---------------------------------------------------------------------- main warps
// A thread's two channels: neighbours in aligned tiles, 32 apart in shifted rows.
template <typename T, bool ROWS, bool DOCS, bool BWD>
struct Main {
    typedef Shape<T, ROWS, BWD> H;
    typedef typename PairWord<T>::type W;
    static constexpr int SEG = H::SEG, kApart = ROWS ? 32 : 1;
    const GateScanArgs& a;
    Shared<H::TOK, DOCS>& sh;
    int lane, warp;
    // the tile at hand
    Tile t;
    const int* doc;
    float2* seg;       // the segment's maps, then states
    uint8_t* st;       // its stage, at this thread's segment and channels
    int s0, c0;        // the segment's first token in the tile; the thread's first channel
    bool ok0, ok1;
    bool plain;        // the segment is inside the sequence, and no document starts or ends in it
    uint32_t marks;    // bit k: a document starts at the segment's token k (SEG: at the token after it)
    int final;         // the sequence's last token, counted from the segment's first
    // ROWS: the low bits of the addresses of the tile's first row and of the bytes from one to the next, per operand
    uint32_t low[ROWS ? H::NA : 1], step[ROWS ? H::NA : 1];

    // Tile n of the walk, for one of its visits.
    __device__ __forceinline__ void open(int n, uint8_t* sm) {
        t = sh.tile[n % kRing];
        doc = sh.doc[DOCS ? n % kRing : 0];
        seg = sh.seg[n & 1][warp];
        s0 = warp * SEG;
        c0 = t.group * kCh + (ROWS ? lane : 2 * lane);
        ok0 = c0 < a.width;
        ok1 = c0 + kApart < a.width;
        st = sm + (n % H::NS) * H::STAGE + (ROWS ? s0 / H::P * H::PITCH + lane * H::ES : s0 * H::PITCH + 2 * lane * H::ES);
        if constexpr (ROWS) {
            auto first = [](const void* base, int64_t at) { return (uint32_t)(uintptr_t)base + (uint32_t)at * H::ES; };
            low[0] = first(a.g, t.og);
            low[1] = first(a.x, t.ox);
            step[0] = (uint32_t)a.g_stride * H::ES;
            step[1] = (uint32_t)a.x_stride * H::ES;
            if constexpr (BWD) {
                low[2] = first(a.dy, t.oy);
                step[2] = (uint32_t)a.width * H::ES;
            }
        }
        plain = s0 + SEG <= t.ntok;
        if (DOCS) {
            marks = __ballot_sync(0xffffffffu, lane <= SEG && doc[s0 + lane] >= 0);
            final = a.seqlen - t.t0 < H::TOK + 1 ? (int)(a.seqlen - t.t0) - 1 - s0 : H::TOK + 1;
            plain = marks == 0 && final >= SEG;
        }
    }
    static __device__ __forceinline__ f2 widen(W w) {
        if constexpr (sizeof(T) == 2) return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        else return w;
    }
    static __device__ __forceinline__ W narrow(f2 v) {
        if constexpr (sizeof(T) == 2) {
            const float2 f = un(v);
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
            return *reinterpret_cast<const uint32_t*>(&b);
        } else {
            return v;
        }
    }
    // The segment's first row of an operand, at the thread's channels; `at`: the tile's offset in it.
    template <typename P>
    __device__ __forceinline__ auto mine(P* base, int64_t at, int64_t pitch) const {
        typedef typename std::conditional<std::is_const<P>::value, const T, T>::type E;
        return static_cast<E*>(base) + at + (uint64_t)(uint32_t)s0 * (uint32_t)pitch + lane;
    }
    // Row k, `pitch` bytes apart, from p (one multiply-add: 64-bit sums would cost two instructions a row)
    template <typename P>
    static __device__ __forceinline__ P* row(P* p, int k, uint32_t pitch) {
        return reinterpret_cast<P*>(reinterpret_cast<uint64_t>(p) + (uint64_t)(uint32_t)k * pitch);
    }
    // One element's bits from a 32-bit register (16-bit values of the language pass through conversions first).
    static __device__ __forceinline__ void put_element(T* q, uint32_t v) {
        if constexpr (sizeof(T) == 2) asm volatile("st.global.u16 [%0], %1;" ::"l"(q), "r"(v) : "memory");
        else asm volatile("st.global.u32 [%0], %1;" ::"l"(q), "r"(v) : "memory");
    }
    // ROWS: the thread's two elements from its first one's place
    static __device__ __forceinline__ f2 pair(const uint8_t* q) {
        typedef typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type E;
        const uint32_t lo = *reinterpret_cast<const E*>(q), hi = *reinterpret_cast<const E*>(q + kApart * H::ES);
        if constexpr (sizeof(T) == 2) return pk(__uint_as_float(lo << 16), __uint_as_float(hi << 16));
        else return pk(__uint_as_float(lo), __uint_as_float(hi));
    }
    // whether the segment's tokens and the tile's channels all exist
    __device__ __forceinline__ bool all() const { return s0 + SEG <= t.ntok && (t.group + 1) * kCh <= a.width; }
    // operand r (g, x, dy) at token k of the segment
    __device__ __forceinline__ f2 in(int r, int k) const {
        if constexpr (ROWS)
            return pair(st + r * H::ARR + (k % H::P * (H::TOK / H::P) + k / H::P) * H::PITCH + ((low[r] + k % H::P * step[r]) & 15));
        else
            return widen(*reinterpret_cast<const W*>(st + r * H::ARR + k * H::PITCH));
    }
    // A result over operand r's place in the stage, from where it is sent off; ROWS: straight to memory, to row k of
    // `base` (the segment's first row, at the thread's channels).
    template <bool ALL>
    __device__ __forceinline__ void put(int r, T* base, int64_t pitch, int k, f2 v) const {
        const W w = narrow(v);
        if constexpr (!ROWS) {
            *reinterpret_cast<W*>(st + r * H::ARR + k * H::PITCH) = w;
        } else {
            T* q = row(base, k, (uint32_t)pitch * H::ES);
            uint32_t lo, hi;
            if constexpr (sizeof(T) == 2) {
                lo = w;
                hi = w >> 16;
            } else {
                const float2 f = un(w);
                lo = __float_as_uint(f.x);
                hi = __float_as_uint(f.y);
            }
            if (ALL || ok0) put_element(q, lo);
            if (ALL || ok1) put_element(q + kApart, hi);
        }
    }
    // two channels of row `row` of a (rows, width) fp32 array, zero without one
    __device__ __forceinline__ f2 state(const float* p, int64_t row) const {
        if (!p) return pk(0.f, 0.f);
        p += row * a.width + c0;
        return pk(ok0 ? __ldg(p) : 0.f, ok1 ? __ldg(p + kApart) : 0.f);
    }
    __device__ __forceinline__ void put_state(float* p, int64_t row, f2 v) const {
        const float2 f = un(v);
        p += row * a.width + c0;
        if (ok0) p[0] = f.x;
        if (ok1) p[kApart] = f.y;
    }
    __device__ __forceinline__ void put_map(f2 A, f2 B) const {
        const float2 fa = un(A), fb = un(B);
        float2* q = seg;
        if constexpr (ROWS) {
            q[lane] = make_float2(fa.x, fb.x);
            q[lane + 32] = make_float2(fa.y, fb.y);
        } else {
            *reinterpret_cast<float4*>(q + 2 * lane) = make_float4(fa.x, fb.x, fa.y, fb.y);
        }
    }
    __device__ __forceinline__ f2 entered() const {
        const float2* q = seg;
        if constexpr (ROWS) return pk(q[lane].x, q[lane + 32].x);
        const float4 e = *reinterpret_cast<const float4*>(q + 2 * lane);
        return pk(e.x, e.z);
    }
    __device__ __forceinline__ bool starts(int k) const { return DOCS && (marks >> k & 1); }
    // whether token k of the segment ends a document, and which
    __device__ __forceinline__ bool ends(int k) const { return DOCS && ((marks >> (k + 1) & 1) || k == final); }
    __device__ __forceinline__ int ending(int k) const { return k == final ? a.ndocs - 1 : doc[s0 + k + 1] - 1; }

    // What the first visit keeps for the second, in registers beside the operands in the stage: e = exp(-g) and,
    // backwards, u = d(h_t)/d(g_t).  ROWS, forwards: a in place of e and u = m x, which reading x again would cost more
    // than its registers.
    struct Keep {
        f2 e[SEG], u[BWD || ROWS ? SEG : 1];
    };

    // PLAIN: every token of the segment is inside the sequence, and no document starts or ends in it
    template <bool PLAIN>
    __device__ __forceinline__ void first_fwd(Keep& q) {
        f2 A = pk(1.f, 1.f), B = pk(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < SEG; ++k) {
            if (!PLAIN && s0 + k >= t.ntok) break;
            const f2 e = forget2(in(0, k)), av = decay2(e);
            if (!PLAIN && starts(k)) {
                A = pk(0.f, 0.f);
                B = state(a.init, doc[s0 + k]);
            }
            A = mul(A, av);
            const f2 b = mul(mul(e, av), in(1, k));
            B = fma2(av, B, b);
            q.e[k] = ROWS ? av : e;
            if constexpr (ROWS) q.u[k] = b;
        }
        put_map(A, B);
    }
    // ALL: the tile's channels all exist
    template <bool PLAIN, bool ALL>
    __device__ __forceinline__ void second_fwd(const Keep& q) {
        f2 h = entered();
        T* y = mine(a.y, t.oy, a.width);
#pragma unroll
        for (int k = 0; k < SEG; ++k) {
            if (!PLAIN && s0 + k >= t.ntok) break;
            if (!PLAIN && starts(k)) h = state(a.init, doc[s0 + k]);
            f2 av, b;
            if constexpr (ROWS) {
                av = q.e[k];
                b = q.u[k];
            } else {
                av = decay2(q.e[k]);
                b = mul(mul(q.e[k], av), in(1, k));
            }
            h = fma2(av, h, b);
            put<ALL>(1, y, a.width, k, h);
            if (DOCS && !PLAIN && a.leave && ends(k)) {
                const int at = ending(k);
                if (at >= 0) put_state(a.leave, at, h);
            }
        }
    }
    template <bool PLAIN>
    __device__ __forceinline__ void first_bwd(Keep& q) {
        const f2 minus = pk(-1.f, -1.f);
        f2 h;
        if (t.t0 + s0 == 0) h = DOCS ? pk(0.f, 0.f) : state(a.init, t.row);
        else if constexpr (ROWS)
            h = pair(st - s0 / H::P * H::PITCH + H::NA * H::ARR + warp * H::PITCH +
                     (((uint32_t)(uintptr_t)a.y + (uint32_t)(t.oy - a.width) * H::ES) & 15));
        else h = widen(*reinterpret_cast<const W*>(st - s0 * H::PITCH + H::NA * H::ARR + warp * H::PITCH));
        // Forwards through the segment: u = (h_{t-1} - x) a (1 - a), and the map of mu over the tokens so far, which the
        // next one's extends from its far end: A is the product of their decays, B the sum of A dy.  A document that ends cuts it.
        f2 A = pk(1.f, 1.f), B = pk(0.f, 0.f);
        bool cut = false;
#pragma unroll
        for (int k = 0; k < SEG; ++k) {
            if (!PLAIN && s0 + k >= t.ntok) break;
            const f2 xv = in(1, k), e = forget2(in(0, k)), av = decay2(e), mv = mul(e, av);
            if (!PLAIN && starts(k)) h = state(a.init, doc[s0 + k]);
            q.u[k] = mul(fma2(xv, minus, h), mul(av, mv));
            q.e[k] = e;
            h = fma2(av, h, mul(mv, xv));
            if (!PLAIN && cut) continue;
            A = mul(A, av);
            B = fma2(A, in(2, k), B);
            if (!PLAIN && ends(k)) {
                const int at = ending(k);
                if (at >= 0) B = fma2(A, state(a.enter, at), B);
                A = pk(0.f, 0.f);
                cut = true;
            }
        }
        put_map(A, B);
    }
    template <bool PLAIN, bool ALL>
    __device__ __forceinline__ void second_bwd(const Keep& q) {
        f2 mu = entered();
        T *dg = mine(a.dg, t.og, a.g_stride), *dx = mine(a.dx, t.ox, a.x_stride);
#pragma unroll
        for (int k = SEG - 1; k >= 0; --k) {
            if (!PLAIN && s0 + k >= t.ntok) continue;
            if (!PLAIN && ends(k)) {
                const int at = ending(k);
                mu = at >= 0 ? state(a.enter, at) : pk(0.f, 0.f);
            }
            const f2 lam = add(in(2, k), mu), av = decay2(q.e[k]), mv = mul(q.e[k], av);
            put<ALL>(0, dg, a.g_stride, k, mul(lam, q.u[k]));
            put<ALL>(1, dx, a.x_stride, k, mul(lam, mv));
            mu = mul(av, lam);
            if (DOCS && !PLAIN && a.leave && starts(k)) put_state(a.leave, doc[s0 + k], mu);
        }
    }

    // The first visit to tile n; false: there is none, or a wait ran out.
    __device__ __forceinline__ bool first(int n, uint8_t* sm, Keep& q) {
        if (!bar_wait(sh, a, &sh.full[n % H::NS], (n / H::NS) & 1, kWhereStage)) return false;
        open(n, sm);
        if (t.ntok) {
            if constexpr (BWD) {
                if (plain) first_bwd<true>(q);
                else first_bwd<false>(q);
            } else {
                if (plain) first_fwd<true>(q);
                else first_fwd<false>(q);
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.maps[n & 1]);
        return t.ntok != 0;
    }
    __device__ __forceinline__ bool second(int n, uint8_t* sm, const Keep& q) {
        if (!bar_wait(sh, a, &sh.states[n & 1], (n >> 1) & 1, kWhereState)) return false;
        open(n, sm);
        if constexpr (BWD) {
            if (plain && (!ROWS || all())) second_bwd<true, true>(q);
            else second_bwd<false, false>(q);
        } else {
            if (plain && (!ROWS || all())) second_fwd<true, true>(q);
            else second_fwd<false, false>(q);
        }
        if (!ROWS) ptx::fence_proxy_async();   // the outputs in the stage, before they are sent off
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.done[n % H::NS]);
        return true;
    }
    __device__ __forceinline__ void run(uint8_t* sm) {
        Keep cur, next;
        bool more = first(0, sm, cur);
        for (int n = 0; more; ++n) {
            more = first(n + 1, sm, next);
            if (!second(n, sm, cur)) return;
            cur = next;
        }
    }
};

template <typename T, bool ROWS, bool DOCS, bool BWD>
__global__ void __launch_bounds__(kThreads, 1) ssd_gate_scan_kernel(const __grid_constant__ ScanParams<T, ROWS, BWD> p) {
    typedef Shape<T, ROWS, BWD> H;
    static_assert(H::kSmem + sizeof(Shared<H::TOK, DOCS>) <= 227 * 1024, "a CTA's shared memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 127) & ~(uintptr_t)127);
    __shared__ __align__(16) Shared<H::TOK, DOCS> sh;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(&sh.full[i], 1);
            ptx::mbar_init(&sh.done[i], kMain);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sh.maps[i], kMain);
            ptx::mbar_init(&sh.told[i], 1);
            ptx::mbar_init(&sh.states[i], 2);
        }
        sh.abort = 0;
        sh.never = 0;
        ptx::mbar_fence_init();
    }
    __syncthreads();
    // The workspace is being cleared by the launch before, which this one does not wait for to start.  Every warp waits here:
    // the main ones read states, and that the clearing has seen what earlier work wrote to them does not make it visible here.
    // It does not let its own successor start early: a clearing that waits on the SMs costs 65536 x 2048 2 us.
    pdl_wait();
    if (warp < kMain) {
        Main<T, ROWS, DOCS, BWD> m = {p.a, sh, (int)(threadIdx.x & 31), warp};
        m.run(sm);
    } else if (warp < kMain + 2) {
        take_states<BWD>(p.a, sh);
    } else if (warp == kMain + 2) {
        publish_maps<BWD>(p.a, sh);
    } else {
        if (DOCS && blockIdx.x == 0) check_cu_seqlens(p.a.cu, p.a.ndocs, p.a.seqlen, p.a.ws, threadIdx.x & 31, 32);
        loading<T, ROWS, DOCS, BWD>(p, sm, sh);
    }
}

__global__ void __launch_bounds__(256) ssd_gate_scan_clear(uint4* p, size_t words) {
    pdl_wait();      // (in this order: this launch's end is then the end of all before it)
    pdl_trigger();
    for (size_t k = (size_t)blockIdx.x * 256 + threadIdx.x; k < words; k += (size_t)gridDim.x * 256) p[k] = make_uint4(0, 0, 0, 0);
}

// One token per batch row: V channels per thread.
template <typename T, int V>
__global__ void __launch_bounds__(256) ssd_gate_scan_step_kernel(GateStepArgs a) {
    pdl_trigger();
    pdl_wait();
    const int per_row = (a.width + V - 1) / V;
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= a.batch * per_row) return;
    const int64_t b = k / per_row;
    const int c = (int)(k - b * per_row) * V;
    Raw<T, V> gr, xr;
    Raw<float, V> sr;
    gr.load(static_cast<const T*>(a.g) + b * a.g_stride + c);
    xr.load(static_cast<const T*>(a.x) + b * a.x_stride + c);
    sr.load(a.state_in + b * a.width + c);
    float g[V], x[V], h[V];
    gr.get(g);
    xr.get(x);
    sr.get(h);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float e = expf(min_nan(-g[j], 87.f)), a = 1.f / (1.f + e);
        h[j] = fmaf(a, h[j], e * a * x[j]);
    }
    sr.set(h);
    sr.store(a.state_out + b * a.width + c);
    Raw<T, V> yr;
    yr.set(h);
    yr.store(static_cast<T*>(a.y) + b * a.width + c);
}

bool on(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

// A (batch, seqlen, width) tensor of token stride `stride`, in boxes of kCh channels x `tokens`, of which every
// `every`-th is read.
bool encode_3d(CUtensorMap* tm, const void* base, int es, const GateScanArgs& a, int64_t stride, int tokens, int every = 1) {
    const auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)a.width, (cuuint64_t)a.seqlen, (cuuint64_t)a.batch};
    cuuint64_t strides[2] = {(cuuint64_t)(stride * es), (cuuint64_t)(a.seqlen * stride * es)};
    cuuint32_t box[3] = {(cuuint32_t)kCh, (cuuint32_t)tokens, 1};
    cuuint32_t step[3] = {1, (cuuint32_t)every, 1};
    return enc(tm, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base),
               dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool ROWS, bool DOCS, bool BWD>
cudaError_t launch_one(const ScanParams<T, ROWS, BWD>& p, cudaStream_t st) {
    const auto kern = ssd_gate_scan_kernel<T, ROWS, DOCS, BWD>;
    constexpr size_t smem = Shape<T, ROWS, BWD>::kSmem;
    // once per device and kernel: the shared-memory opt-in
    static std::atomic<uint8_t> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
        ready[dev].store(1, std::memory_order_release);
    }
    // one CTA per SM; with tickets any number of them finishes the work
    const int nsm = device_sms();
    const uint32_t most = nsm > 0 ? nsm : 152;
    return launch_kernel(kern, p.a.ntiles < most ? p.a.ntiles : most, kThreads, smem, st, p.a.ws != nullptr, p);
}

// Class k of P of a matrix's rows (its rows k, k + P, ...), in boxes of kCh + P columns x `box` rows.  Its rows are aligned as
// its first one is, and are read from the 16-byte boundary before it.  A class without rows is not looked at; its
// map holds the first row.
template <typename T>
bool encode_class(CUtensorMap* tm, const void* base, int64_t rows, int width, int64_t stride, int k, int box) {
    constexpr int es = sizeof(T), P = 16 / es;
    const auto enc = tensor_map_encoder();
    if (!enc) return false;
    const uintptr_t at = (uintptr_t)base + (k < rows ? (uintptr_t)k * stride * es : 0), from = at & ~(uintptr_t)15;
    const int64_t n = k < rows ? (rows - k + P - 1) / P : 1;
    cuuint64_t dims[2] = {(cuuint64_t)(width + (at - from) / es), (cuuint64_t)n};
    // a single row has no stride, and that of several is within the memory that they lie in
    cuuint64_t strides[1] = {(cuuint64_t)(n > 1 ? stride : width + P) * es * P};
    cuuint32_t boxes[2] = {(cuuint32_t)(kCh + P), (cuuint32_t)box};
    cuuint32_t step[2] = {1, 1};
    return enc(tm, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, reinterpret_cast<void*>(from),
               dims, strides, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool BWD>
cudaError_t launch_rows(const GateScanArgs& a, cudaStream_t st) {
    typedef Shape<T, true, BWD> H;
    ScanParams<T, true, BWD> p;
    p.a = a;
    const int64_t rows = a.batch * a.seqlen;
    for (int k = 0; k < H::P; ++k) {
        const int box = H::TOK / H::P;
        bool ok = encode_class<T>(&p.g[k], a.g, rows, a.width, a.g_stride, k, box) &&
                  encode_class<T>(&p.x[k], a.x, rows, a.width, a.x_stride, k, box);
        if constexpr (BWD)
            ok = ok && encode_class<T>(&p.dy[k], a.dy, rows, a.width, a.width, k, box) &&
                 encode_class<T>(&p.y[k], a.y, rows, a.width, a.width, k, kMain);
        if (!ok) return cudaErrorInvalidValue;
    }
    return a.cu ? launch_one<T, true, true, BWD>(p, st) : launch_one<T, true, false, BWD>(p, st);
}

template <typename T, bool BWD>
cudaError_t launch_typed(const GateScanArgs& a, bool rows, cudaStream_t st) {
    if (rows) return launch_rows<T, BWD>(a, st);
    ScanParams<T, false, BWD> p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    typedef Shape<T, false, BWD> H;
    constexpr int es = sizeof(T);
    bool ok = encode_3d(&p.g, a.g, es, a, a.g_stride, H::TOK) && encode_3d(&p.x, a.x, es, a, a.x_stride, H::TOK) &&
              encode_3d(&p.y, a.y, es, a, a.width, H::TOK, BWD ? H::SEG : 1);
    if (BWD)
        ok = ok && encode_3d(&p.dy, a.dy, es, a, a.width, H::TOK) && encode_3d(&p.dg, a.dg, es, a, a.g_stride, H::TOK) &&
             encode_3d(&p.dx, a.dx, es, a, a.x_stride, H::TOK);
    if (!ok) return cudaErrorInvalidValue;
    return a.cu ? launch_one<T, false, true, BWD>(p, st) : launch_one<T, false, false, BWD>(p, st);
}

// Whether rows can be moved as TMA tiles: every row of every operand starts on a 16-byte boundary.
bool aligned_rows(const GateScanArgs& a, bool bwd) {
    const int unit = a.dtype == SSD_BF16 ? 8 : 4;
    if (a.width % unit || a.g_stride % unit || a.x_stride % unit || !on(a.g, 16) || !on(a.x, 16) || !on(a.y, 16)) return false;
    // a tensor map's strides are below 2^40 bytes
    const int64_t most = ((int64_t)1 << 40) / a.seqlen / 4;
    if (a.g_stride >= most || a.x_stride >= most) return false;
    return !bwd || (on(a.dy, 16) && on(a.dg, 16) && on(a.dx, 16));
}

GateScanLayout layout(int64_t batch, int64_t seqlen, int width, int dtype, bool bwd, bool rows) {
    GateScanLayout l;
    const int tok = scan_seg(bwd, dtype, rows) * kMain;
    l.nchunks = (seqlen + tok - 1) / tok;
    l.ngroups = (width + kCh - 1) / kCh;
    l.nblocks = (l.nchunks + kBlock - 1) / kBlock;
    const size_t lines = (size_t)batch * l.ngroups;
    l.ticket_off = sizeof(WsHeader);
    l.maps_off = l.ticket_off + 256;
    l.carry_off = l.maps_off + lines * l.nchunks * kCh * 8;
    l.total = l.carry_off + lines * l.nblocks * kCh * 8;
    if (l.nchunks == 1) l.total = sizeof(WsHeader);
    return l;
}

}  // namespace

size_t gate_scan_workspace(int64_t batch, int64_t seqlen, int width, int dtype) {
    size_t most = 0;
    for (int k = 0; k < 4; ++k) {
        const size_t t = layout(batch, seqlen, width, dtype, k & 1, k & 2).total;
        if (t > most) most = t;
    }
    return most;
}

cudaError_t launch_gate_scan(const GateScanArgs& args, void* workspace, bool bwd, cudaStream_t st) {
    GateScanArgs a = args;
    const bool rows = !aligned_rows(a, bwd);
    const GateScanLayout l = layout(a.batch, a.seqlen, a.width, a.dtype, bwd, rows);
    char* w = static_cast<char*>(workspace);
    a.nchunks = l.nchunks;
    a.ngroups = l.ngroups;
    a.nblocks = l.nblocks;
    a.ntiles = (uint32_t)(a.batch * l.ngroups * l.nchunks);
    if (a.wait_iters == 0) {
        a.wait_iters = kDefaultWaitIters;
        a.loads = -1;
    }
    a.ws = reinterpret_cast<WsHeader*>(w);
    a.ticket = reinterpret_cast<uint32_t*>(w + l.ticket_off);
    a.maps = reinterpret_cast<uint64_t*>(w + l.maps_off);
    a.carry = reinterpret_cast<uint64_t*>(w + l.carry_off);
    // status word, tickets, maps and carried states start from zero
    if (workspace) {
        const size_t words = l.total / 16, ctas = (words + 1023) / 1024;
        const cudaError_t e = launch_kernel(ssd_gate_scan_clear, (unsigned)(ctas < 304 ? ctas : 304), 256, 0, st, true,
                                            static_cast<uint4*>(workspace), words);
        if (e != cudaSuccess) return e;
    }
    if (a.dtype == SSD_BF16) return bwd ? launch_typed<bf16_t, true>(a, rows, st) : launch_typed<bf16_t, false>(a, rows, st);
    return bwd ? launch_typed<float, true>(a, rows, st) : launch_typed<float, false>(a, rows, st);
}

cudaError_t launch_gate_scan_step(const GateStepArgs& a, cudaStream_t st) {
    const size_t e = a.dtype == SSD_BF16 ? 2 : 4;
    const bool vec = a.width % 4 == 0 && a.g_stride % 4 == 0 && a.x_stride % 4 == 0 && on(a.g, 4 * e) && on(a.x, 4 * e) &&
                     on(a.y, 4 * e) && on(a.state_in, 16) && on(a.state_out, 16);
    const int64_t n = a.batch * ((a.width + (vec ? 3 : 0)) / (vec ? 4 : 1));
    const unsigned grid = (unsigned)((n + 255) / 256);
    void (*const kern)(GateStepArgs) =
        a.dtype == SSD_BF16 ? (vec ? ssd_gate_scan_step_kernel<bf16_t, 4> : ssd_gate_scan_step_kernel<bf16_t, 1>)
                            : (vec ? ssd_gate_scan_step_kernel<float, 4> : ssd_gate_scan_step_kernel<float, 1>);
    return launch_kernel(kern, grid, 256, 0, st, true, a);
}

}  // namespace ssd
