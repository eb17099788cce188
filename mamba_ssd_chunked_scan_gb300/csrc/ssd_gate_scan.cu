// Gated linear recurrence, one decay per channel and token:
//   ssd_gate_scan_kernel       h_t = a_t h_{t-1} + (1 - a_t) x_t,  a_t = 1 / (1 + exp(-g_t)),  y = h
//   ssd_gate_scan_bwd_kernel   lam_t = dy_t + a_{t+1} lam_{t+1};  dx = (1 - a) lam,
//                              dg = lam (h_{t-1} - x) a (1 - a),  dinit = a_1 lam_1
//   ssd_gate_scan_step_kernel  one token from a resident state
//
// Each step is an affine map of the state, and the maps of consecutive steps
// compose: (A2, B2) o (A1, B1) = (A2 A1, A2 B1 + B2).  A CTA takes one tile of
// kTok tokens x kCh channels: a warp holds a segment of kSeg tokens, a thread two
// channels of it, with the tile's decays and inputs in registers from their one
// read to the one write of y.  A tile needs the state that enters it.  Its map
// is published as soon as it is known; the state follows from the maps of the
// tiles before it in its block of kBlock tiles and from the state that enters the
// block, which the last tile of the block before publishes.  So only one hand-over
// per block is a chain, every input is read once, and the order in which maps are
// composed is fixed: results do not depend on which tile ran first.  Tiles are
// taken by ticket in the order of the sequence (a tile only waits for tiles
// with smaller tickets, which running CTAs hold), and every wait is bounded.
//
// The backward pass walks the same maps from the end: mu_t = a_t lam_t obeys
// mu_t = a_t (dy_t + mu_{t+1}).  h_{t-1} inside a segment is recomputed from
// the h before it, which is read from y (rounded to y's type once, at every
// kSeg-th token); keeping every h would cost as many bytes again as g.
//
// A document's first token cuts the map (A = 0) and takes the document's own state.
//
// 1 - a is formed as e / (1 + e), e = exp(-g), not as a difference: a channel
// with a long memory has a close to 1.
#include "ssd_common.cuh"
#include "ssd_kernels.h"
#include "ssd_vec.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

constexpr int kSeg = 16;               // tokens per segment (one warp)
constexpr int kWarps = kScanTok / kSeg;
constexpr int kThreads = 32 * kWarps;
constexpr int kCh = kScanCh;           // channels per tile: two per thread
constexpr int kTok = kScanTok;
constexpr int kBlock = kScanBlock;

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kWhereTile = 51, kWhereBlock = 52;

// a = 1 / (1 + e), m = e / (1 + e) with e = exp(-g), capped where e would overflow
// (a is then 1e-38, m one).  bf16 operands take the special-function unit's
// approximations (relative error of a few 2^-23); fp32 ones the rounded forms.
template <typename T>
__device__ __forceinline__ void gate(float g, float& a, float& m) {
    if constexpr (sizeof(T) == 2) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fminf(-g * kLog2e, 126.f)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(1.f + e));
        m = e * a;
    } else {
        const float e = expf(fminf(-g, 87.f));
        a = __frcp_rn(1.f + e);
        m = e * a;
    }
    if (g != g) a = m = g;   // fminf drops a NaN
}

// The two channels of a thread: neighbours (one access) where rows allow it, else
// 32 apart (two accesses, each contiguous over the warp).
template <typename T, bool PAIR>
struct Two {
    T lo, hi;   // as stored
    __device__ __forceinline__ void load(const T* p, bool ok0, bool ok1) {
        if constexpr (PAIR) {
            Raw<T, 2> r;
            r.zero();
            if (ok0) r.load(p);
            const T* e = reinterpret_cast<const T*>(&r.w);
            lo = e[0];
            hi = e[1];
        } else {
            Raw<T, 1> r, q;
            r.zero();
            q.zero();
            if (ok0) r.load(p);
            if (ok1) q.load(p + 32);
            lo = *reinterpret_cast<const T*>(&r.w);
            hi = *reinterpret_cast<const T*>(&q.w);
        }
    }
    static __device__ __forceinline__ void store(T* p, bool ok0, bool ok1, float v0, float v1) {
        if constexpr (PAIR) {
            const float v[2] = {v0, v1};
            Raw<T, 2> r;
            r.set(v);
            if (ok0) r.store(p);
        } else {
            const float a[1] = {v0}, b[1] = {v1};
            Raw<T, 1> r, q;
            r.set(a);
            q.set(b);
            if (ok0) r.store(p);
            if (ok1) q.store(p + 32);
        }
    }
    __device__ __forceinline__ float f0() const { return (float)lo; }
    __device__ __forceinline__ float f1() const { return (float)hi; }
};

struct Tile {
    int64_t row, chunk;    // batch row, tile along the sequence
    int64_t t0;            // its first token
    int group;             // channel group
    int ntok;              // its tokens
};

// Documents that start inside the tile (or at the token after it): doc[k] = the
// document that starts at token t0 + k, or -1.  Offsets outside the tile are skipped,
// so nothing they hold can index out of bounds.
__device__ void find_docs(const GateScanArgs& a, int64_t t0, int* doc) {
    for (int k = threadIdx.x; k <= kTok; k += kThreads) doc[k] = -1;
    __syncthreads();
    // the first document whose offset is >= t0
    int lo = 0, hi = a.ndocs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) < t0) lo = mid + 1;
        else hi = mid;
    }
    for (int d = lo + threadIdx.x; d < a.ndocs; d += kThreads) {
        const int64_t k = (int64_t)__ldg(a.cu + d) - t0;
        if (k > kTok) break;
        if (k >= 0) doc[k] = d;
    }
    __syncthreads();
}

struct Maps {   // a segment's map per channel
    float2 A[kWarps][32], B[kWarps][32];
};

// The maps of the tile's predecessors in its block, and the state that enters the block.
struct Before {
    float2 A[kBlock][32], B[kBlock][32];
    float2 carry[32];
    int ok;
};

__device__ __forceinline__ bool wait_flag(const uint32_t* flag, WsHeader* ws, uint32_t where) {
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t it = 0;; ++it) {
        uint32_t v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v) return true;
        if ((it & 63) == 63 && (ptx::globaltimer() - t0 > kWaitNs || it > (1u << 26))) {
            record_error(ws, SSD_ERR_TIMEOUT, where);
            return false;
        }
    }
}
__device__ __forceinline__ void raise_flag(uint32_t* flag) {
    asm volatile("st.release.gpu.global.u32 [%0], 1;" ::"l"(flag) : "memory");
}

// Takes the next tile in sequence order (tickets), or the CTA's own where the call
// has one tile per sequence.
template <bool REV>
__device__ bool take_tile(const GateScanArgs& a, Tile& t, int* slot) {
    uint32_t k = blockIdx.x;
    if (a.nchunks > 1) {
        if (threadIdx.x == 0) *slot = (int)atomicAdd(a.ticket, 1u);
        __syncthreads();
        k = (uint32_t)*slot;
    }
    const uint32_t per = (uint32_t)(a.batch * a.ngroups);
    const uint32_t c = k / per, r = k - c * per;
    t.row = r / (uint32_t)a.ngroups;
    t.group = (int)(r - (uint32_t)t.row * a.ngroups);
    t.chunk = REV ? a.nchunks - 1 - c : c;
    t.t0 = t.chunk * kTok;
    t.ntok = (int)((a.seqlen - t.t0 < kTok) ? a.seqlen - t.t0 : kTok);
    return true;
}

// Publishes the tile's map and returns the value that enters it, per channel: `init`
// enters the sequence's first tile.  `step` is the tile's place in the order
// of the walk.  Called by every thread; the map (A, B) of the whole tile is valid in warp 0.
__device__ float2 enter_tile(const GateScanArgs& a, const Tile& t, int64_t step, float2 A, float2 B, float2 init, Before& bf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (a.nchunks == 1) return init;
    const int64_t line = t.row * a.ngroups + t.group;         // sequence of tiles
    const int64_t base = line * a.nchunks;                    // its first slot
    const int in_block = (int)(step % kBlock);
    const int64_t block = step / kBlock;
    const int64_t nblocks = (a.nchunks + kBlock - 1) / kBlock;
    if (warp == 0 && in_block != kBlock - 1 && step != a.nchunks - 1) {
        a.maps[(base + step) * 32 + lane] = make_float4(A.x, A.y, B.x, B.y);
        __threadfence();
        __syncwarp();
        if (lane == 0) raise_flag(a.map_flag + base + step);
    }
    if (threadIdx.x == 0) bf.ok = 1;
    __syncthreads();
    // warp w fetches the maps of predecessors w, w + kWarps, ...; the last warp the carry
    for (int p = warp; p < in_block; p += kWarps) {
        bool ok = true;
        if (lane == 0) ok = wait_flag(a.map_flag + base + block * kBlock + p, a.ws, kWhereTile);
        if (!ok) bf.ok = 0;
        __syncwarp();
        const float4 m = __ldcg(a.maps + (base + block * kBlock + p) * 32 + lane);
        bf.A[p][lane] = make_float2(m.x, m.y);
        bf.B[p][lane] = make_float2(m.z, m.w);
    }
    if (warp == kWarps - 1) {
        float2 c = init;
        if (block > 0) {
            bool ok = true;
            if (lane == 0) ok = wait_flag(a.carry_flag + line * nblocks + block - 1, a.ws, kWhereBlock);
            if (!ok) bf.ok = 0;
            __syncwarp();
            c = __ldcg(a.carry + (line * nblocks + block - 1) * 32 + lane);
        }
        bf.carry[lane] = c;
    }
    __syncthreads();
    float2 h = bf.carry[lane];
    for (int p = 0; p < in_block; ++p) {
        h.x = fmaf(bf.A[p][lane].x, h.x, bf.B[p][lane].x);
        h.y = fmaf(bf.A[p][lane].y, h.y, bf.B[p][lane].y);
    }
    if (warp == 0 && in_block == kBlock - 1 && step != a.nchunks - 1) {
        a.carry[(line * nblocks + block) * 32 + lane] = make_float2(fmaf(A.x, h.x, B.x), fmaf(A.y, h.y, B.y));
        __threadfence();
        __syncwarp();
        if (lane == 0) raise_flag(a.carry_flag + line * nblocks + block);
    }
    return h;
}

// The map of segments [from, to) (in the walk's order), composed in order.
template <bool REV>
__device__ __forceinline__ void compose(const Maps& mp, int n, int lane, float2& A, float2& B) {
    A = make_float2(1.f, 1.f);
    B = make_float2(0.f, 0.f);
    for (int k = 0; k < n; ++k) {
        const int w = REV ? kWarps - 1 - k : k;
        const float2 a = mp.A[w][lane], b = mp.B[w][lane];
        B.x = fmaf(a.x, B.x, b.x);
        B.y = fmaf(a.y, B.y, b.y);
        A.x *= a.x;
        A.y *= a.y;
    }
}

template <typename T, bool PAIR, bool DOCS>
__global__ void __launch_bounds__(kThreads) ssd_gate_scan_kernel(GateScanArgs a) {
    __shared__ Maps mp;
    __shared__ Before bf;
    __shared__ int doc[DOCS ? kTok + 1 : 1];
    __shared__ int slot;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Tile t;
    take_tile<false>(a, t, &slot);
    if (DOCS) {
        find_docs(a, t.t0, doc);
        if (blockIdx.x == 0) check_cu_seqlens(a.cu, a.ndocs, a.seqlen, a.ws, threadIdx.x, kThreads);
    }
    const int c0 = t.group * kCh + (PAIR ? 2 * lane : lane), c1 = c0 + (PAIR ? 1 : 32);
    const bool ok0 = c0 < a.width, ok1 = c1 < a.width;
    const int s0 = warp * kSeg;   // first token of the segment in the tile
    const int64_t tok = t.row * a.seqlen + t.t0 + s0;
    const T* g = static_cast<const T*>(a.g) + tok * a.g_stride + c0;
    const T* x = static_cast<const T*>(a.x) + tok * a.x_stride + c0;
    Two<T, PAIR> gr[kSeg], xr[kSeg];
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        const bool in = s0 + k < t.ntok;
        gr[k].load(g + k * a.g_stride, ok0 && in, ok1 && in);
        xr[k].load(x + k * a.x_stride, ok0 && in, ok1 && in);
    }
    // the segment's map; its decays and inputs stay in registers
    float2 av[kSeg], bv[kSeg];
    float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        if (s0 + k >= t.ntok) {   // past the sequence's end: the identity
            av[k] = make_float2(1.f, 1.f);
            bv[k] = make_float2(0.f, 0.f);
            continue;
        }
        float m0, m1;
        gate<T>(gr[k].f0(), av[k].x, m0);
        gate<T>(gr[k].f1(), av[k].y, m1);
        bv[k] = make_float2(m0 * xr[k].f0(), m1 * xr[k].f1());
        if (DOCS && doc[s0 + k] >= 0) {
            const float* in = a.init ? a.init + (int64_t)doc[s0 + k] * a.width + c0 : nullptr;
            if (in && ok0) bv[k].x = fmaf(av[k].x, __ldg(in), bv[k].x);
            if (in && ok1) bv[k].y = fmaf(av[k].y, __ldg(in + c1 - c0), bv[k].y);
            av[k] = make_float2(0.f, 0.f);
        }
        B.x = fmaf(av[k].x, B.x, bv[k].x);
        B.y = fmaf(av[k].y, B.y, bv[k].y);
        A.x *= av[k].x;
        A.y *= av[k].y;
    }
    mp.A[warp][lane] = A;
    mp.B[warp][lane] = B;
    __syncthreads();
    float2 init = make_float2(0.f, 0.f);
    if (!DOCS && a.init) {
        const float* in = a.init + t.row * a.width + c0;
        if (ok0) init.x = __ldg(in);
        if (ok1) init.y = __ldg(in + c1 - c0);
    }
    if (warp == 0) compose<false>(mp, kWarps, lane, A, B);
    float2 h = enter_tile(a, t, t.chunk, A, B, init, bf);
    compose<false>(mp, warp, lane, A, B);
    h.x = fmaf(A.x, h.x, B.x);
    h.y = fmaf(A.y, h.y, B.y);
    T* y = static_cast<T*>(a.y) + tok * a.width + c0;
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        const bool in = s0 + k < t.ntok;
        h.x = fmaf(av[k].x, h.x, bv[k].x);
        h.y = fmaf(av[k].y, h.y, bv[k].y);
        Two<T, PAIR>::store(y + (int64_t)k * a.width, ok0 && in, ok1 && in, h.x, h.y);
        if (a.fin && in) {
            const bool last = t.t0 + s0 + k == a.seqlen - 1;
            int64_t at = -1;
            if (DOCS) at = last ? a.ndocs - 1 : doc[s0 + k + 1] - 1;   // the document before the one that starts next
            else if (last) at = t.row;
            if (at >= 0) {
                float* f = a.fin + at * a.width + c0;
                if (ok0) f[0] = h.x;
                if (ok1) f[c1 - c0] = h.y;
            }
        }
    }
}

template <typename T, bool PAIR, bool DOCS>
__global__ void __launch_bounds__(kThreads) ssd_gate_scan_bwd_kernel(GateScanArgs a) {
    __shared__ Maps mp;
    __shared__ Before bf;
    __shared__ int doc[DOCS ? kTok + 1 : 1];
    __shared__ int slot;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Tile t;
    take_tile<true>(a, t, &slot);
    if (DOCS) {
        find_docs(a, t.t0, doc);
        if (blockIdx.x == 0) check_cu_seqlens(a.cu, a.ndocs, a.seqlen, a.ws, threadIdx.x, kThreads);
    }
    const int c0 = t.group * kCh + (PAIR ? 2 * lane : lane), c1 = c0 + (PAIR ? 1 : 32);
    const bool ok0 = c0 < a.width, ok1 = c1 < a.width;
    const int s0 = warp * kSeg;
    const int64_t tok = t.row * a.seqlen + t.t0 + s0;
    const T* g = static_cast<const T*>(a.g) + tok * a.g_stride + c0;
    const T* x = static_cast<const T*>(a.x) + tok * a.x_stride + c0;
    const T* dy = static_cast<const T*>(a.dy) + tok * a.width + c0;
    Two<T, PAIR> gr[kSeg], xr[kSeg], dr[kSeg], hr;
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        const bool in = s0 + k < t.ntok;
        gr[k].load(g + k * a.g_stride, ok0 && in, ok1 && in);
        xr[k].load(x + k * a.x_stride, ok0 && in, ok1 && in);
        dr[k].load(dy + (int64_t)k * a.width, ok0 && in, ok1 && in);
    }
    // h before the segment: the output before it, or the state that enters the sequence
    const bool first = t.t0 + s0 == 0;
    const bool any = s0 < t.ntok && !first;
    hr.load(static_cast<const T*>(a.y) + (tok - (any ? 1 : 0)) * a.width + c0, ok0 && any, ok1 && any);
    float2 h = make_float2(hr.f0(), hr.f1());
    if (first && !DOCS && a.init) {
        const float* in = a.init + t.row * a.width + c0;
        if (ok0) h.x = __ldg(in);
        if (ok1) h.y = __ldg(in + c1 - c0);
    }
    // forwards through the segment: uv = d(h_t)/d(g_t) = (h_{t-1} - x) a (1 - a), mv = 1 - a
    float2 uv[kSeg], mv[kSeg];
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        float a0, a1;
        const float x0 = xr[k].f0(), x1 = xr[k].f1();
        gate<T>(gr[k].f0(), a0, mv[k].x);
        gate<T>(gr[k].f1(), a1, mv[k].y);
        if (DOCS && s0 + k < t.ntok && doc[s0 + k] >= 0) {
            h = make_float2(0.f, 0.f);
            const float* in = a.init ? a.init + (int64_t)doc[s0 + k] * a.width + c0 : nullptr;
            if (in && ok0) h.x = __ldg(in);
            if (in && ok1) h.y = __ldg(in + c1 - c0);
        }
        const float e0 = h.x - x0, e1 = h.y - x1;
        uv[k].x = e0 * a0 * mv[k].x;
        uv[k].y = e1 * a1 * mv[k].y;
        h.x = fmaf(a0, h.x, mv[k].x * x0);
        h.y = fmaf(a1, h.y, mv[k].y * x1);
    }
    // backwards: the map of mu over the segment.  dfin enters at a document's (or row's) last
    // token, which cuts the map.
    float2 A = make_float2(1.f, 1.f), B = make_float2(0.f, 0.f);
    auto ends = [&](int k) { return DOCS && (doc[s0 + k + 1] >= 0 || t.t0 + s0 + k == a.seqlen - 1); };
    auto dfin_of = [&](int k) {
        float2 d = make_float2(0.f, 0.f);
        const int64_t at = t.t0 + s0 + k == a.seqlen - 1 ? a.ndocs - 1 : doc[s0 + k + 1] - 1;
        if (a.dfin && at >= 0) {
            const float* f = a.dfin + at * a.width + c0;
            if (ok0) d.x = __ldg(f);
            if (ok1) d.y = __ldg(f + c1 - c0);
        }
        return d;
    };
#pragma unroll
    for (int k = kSeg - 1; k >= 0; --k) {
        if (s0 + k >= t.ntok) continue;
        if (DOCS && ends(k)) {
            A = make_float2(0.f, 0.f);
            B = dfin_of(k);
        }
        const float a0 = 1.f - mv[k].x, a1 = 1.f - mv[k].y;
        B.x = a0 * (dr[k].f0() + B.x);
        B.y = a1 * (dr[k].f1() + B.y);
        A.x *= a0;
        A.y *= a1;
    }
    mp.A[warp][lane] = A;
    mp.B[warp][lane] = B;
    __syncthreads();
    float2 last = make_float2(0.f, 0.f);
    if (!DOCS && a.dfin) {
        const float* f = a.dfin + t.row * a.width + c0;
        if (ok0) last.x = __ldg(f);
        if (ok1) last.y = __ldg(f + c1 - c0);
    }
    if (warp == 0) compose<true>(mp, kWarps, lane, A, B);
    float2 mu = enter_tile(a, t, a.nchunks - 1 - t.chunk, A, B, last, bf);
    compose<true>(mp, kWarps - 1 - warp, lane, A, B);
    mu.x = fmaf(A.x, mu.x, B.x);
    mu.y = fmaf(A.y, mu.y, B.y);
    T* dg = static_cast<T*>(a.dg) + tok * a.g_stride + c0;
    T* dx = static_cast<T*>(a.dx) + tok * a.x_stride + c0;
#pragma unroll
    for (int k = kSeg - 1; k >= 0; --k) {
        const bool in = s0 + k < t.ntok;
        if (!in) continue;
        if (DOCS && ends(k)) mu = dfin_of(k);
        const float l0 = dr[k].f0() + mu.x, l1 = dr[k].f1() + mu.y;
        Two<T, PAIR>::store(dg + k * a.g_stride, ok0, ok1, l0 * uv[k].x, l1 * uv[k].y);
        Two<T, PAIR>::store(dx + k * a.x_stride, ok0, ok1, l0 * mv[k].x, l1 * mv[k].y);
        mu.x = (1.f - mv[k].x) * l0;
        mu.y = (1.f - mv[k].y) * l1;
        if (a.dinit) {
            int64_t at = -1;
            if (DOCS) at = doc[s0 + k];
            else if (t.t0 + s0 + k == 0) at = t.row;
            if (at >= 0) {
                float* f = a.dinit + at * a.width + c0;
                if (ok0) f[0] = mu.x;
                if (ok1) f[c1 - c0] = mu.y;
            }
        }
    }
}

// One token per batch row: V channels per thread.
template <typename T, int V>
__global__ void __launch_bounds__(256) ssd_gate_scan_step_kernel(GateStepArgs a) {
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
        float d, m;
        gate<float>(g[j], d, m);
        h[j] = fmaf(d, h[j], m * x[j]);
    }
    sr.set(h);
    sr.store(a.state_out + b * a.width + c);
    Raw<T, V> yr;
    yr.set(h);
    yr.store(static_cast<T*>(a.y) + b * a.width + c);
}

bool on(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

template <typename T, bool BWD>
cudaError_t launch_typed(const GateScanArgs& a, cudaStream_t st) {
    const size_t two = 2 * sizeof(T);
    bool pair = a.width % 2 == 0 && a.g_stride % 2 == 0 && a.x_stride % 2 == 0 && on(a.g, two) && on(a.x, two) && on(a.y, two);
    if (BWD) pair = pair && on(a.dy, two) && on(a.dg, two) && on(a.dx, two);
    const bool docs = a.cu != nullptr;
    void (*kern)(GateScanArgs);
    if (BWD)
        kern = pair ? (docs ? ssd_gate_scan_bwd_kernel<T, true, true> : ssd_gate_scan_bwd_kernel<T, true, false>)
                    : (docs ? ssd_gate_scan_bwd_kernel<T, false, true> : ssd_gate_scan_bwd_kernel<T, false, false>);
    else
        kern = pair ? (docs ? ssd_gate_scan_kernel<T, true, true> : ssd_gate_scan_kernel<T, true, false>)
                    : (docs ? ssd_gate_scan_kernel<T, false, true> : ssd_gate_scan_kernel<T, false, false>);
    const int64_t grid = a.nchunks * a.batch * a.ngroups;
    kern<<<(unsigned)grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

GateScanLayout gate_scan_layout(int64_t batch, int64_t seqlen, int width) {
    GateScanLayout l;
    l.nchunks = (seqlen + kTok - 1) / kTok;
    l.ngroups = (width + kCh - 1) / kCh;
    const size_t lines = (size_t)batch * l.ngroups, nblocks = (size_t)((l.nchunks + kBlock - 1) / kBlock);
    l.ticket_off = sizeof(WsHeader);
    l.map_flag_off = l.ticket_off + 256;
    l.carry_flag_off = l.map_flag_off + lines * l.nchunks * 4;
    l.clear_bytes = align_up(l.carry_flag_off + lines * nblocks * 4, 256);
    l.maps_off = l.clear_bytes;
    l.carry_off = l.maps_off + lines * l.nchunks * 32 * 16;
    l.total = l.carry_off + lines * nblocks * 32 * 8;
    if (l.nchunks == 1) l.total = l.clear_bytes = sizeof(WsHeader);
    return l;
}

cudaError_t launch_gate_scan(const GateScanArgs& args, void* workspace, bool bwd, cudaStream_t st) {
    GateScanArgs a = args;
    const GateScanLayout l = gate_scan_layout(a.batch, a.seqlen, a.width);
    char* w = static_cast<char*>(workspace);
    a.nchunks = l.nchunks;
    a.ngroups = l.ngroups;
    a.ws = reinterpret_cast<WsHeader*>(w);
    a.ticket = reinterpret_cast<uint32_t*>(w + l.ticket_off);
    a.map_flag = reinterpret_cast<uint32_t*>(w + l.map_flag_off);
    a.carry_flag = reinterpret_cast<uint32_t*>(w + l.carry_flag_off);
    a.maps = reinterpret_cast<float4*>(w + l.maps_off);
    a.carry = reinterpret_cast<float2*>(w + l.carry_off);
    // status word, tickets and flags start from zero
    const cudaError_t e = cudaMemsetAsync(workspace, 0, l.clear_bytes, st);
    if (e != cudaSuccess) return e;
    if (a.dtype == SSD_BF16) return bwd ? launch_typed<bf16_t, true>(a, st) : launch_typed<bf16_t, false>(a, st);
    return bwd ? launch_typed<float, true>(a, st) : launch_typed<float, false>(a, st);
}

cudaError_t launch_gate_scan_step(const GateStepArgs& a, cudaStream_t st) {
    const size_t e = a.dtype == SSD_BF16 ? 2 : 4;
    const bool vec = a.width % 4 == 0 && a.g_stride % 4 == 0 && a.x_stride % 4 == 0 && on(a.g, 4 * e) && on(a.x, 4 * e) &&
                     on(a.y, 4 * e) && on(a.state_in, 16) && on(a.state_out, 16);
    const int64_t n = a.batch * ((a.width + (vec ? 3 : 0)) / (vec ? 4 : 1));
    const unsigned grid = (unsigned)((n + 255) / 256);
    if (a.dtype == SSD_BF16) {
        if (vec) ssd_gate_scan_step_kernel<bf16_t, 4><<<grid, 256, 0, st>>>(a);
        else ssd_gate_scan_step_kernel<bf16_t, 1><<<grid, 256, 0, st>>>(a);
    } else {
        if (vec) ssd_gate_scan_step_kernel<float, 4><<<grid, 256, 0, st>>>(a);
        else ssd_gate_scan_step_kernel<float, 1><<<grid, 256, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace ssd
