// Root-mean-square norm with the residual's addition, and its gradient:
//   ssd_add_norm_kernel       h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps),
//                             out = h rstd w  (bf16, fp32, or e4m3 rows with a scale each)
//   ssd_add_norm_bwd_kernel   dh = rstd (w do - xh mean(w do xh)) + dres,  xh = h rstd,
//                             and each row slot's share of dw = sum_rows do xh
//   ssd_add_norm_bwd_reduce   dw from the shares, in a fixed order
//
// A row is held in registers from its one read to its one write, so both passes
// are bound by HBM: 16384 x 2560, bf16 with an fp32 residual, 73.9 us forward (6.81 TB/s), e4m3 rows 69 us;
// 12289 x 2560 backward 80.7 us (6.2 TB/s; a plain copy reaches 6.77).  A row belongs to consecutive threads of a CTA, 16
// elements each (8 or 16 in the backward): as 16-byte vectors of x where the width and the addresses
// allow (in the backward, whatever the width), one by one (strided by the row's threads, so that a warp's accesses
// stay contiguous) where they do not.  Rows that fit a warp take one
// each, several rows to a CTA; longer rows take a CTA.
//
// The sums are fp32; h is normalised as it was summed, before its rounding to the
// residual stream's type.  e4m3: scale = max(max |out|, 1e-30) / 448, and the row
// holds the fp32 quotient out / scale rounded to nearest even; the floor keeps the quotient of an
// all-zero row finite.  The quotient is the product with the reciprocal, corrected by its remainder, which an fma gives
// exactly (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990): a
// product alone would put values beside the midpoint of two e4m3 numbers on the wrong side.
#include "ssd_common.cuh"
#include "ssd_kernels.h"
#include "ssd_vec.cuh"

namespace ssd {
namespace {

constexpr int kElems = 16;      // elements of a row per thread
constexpr int kBwdElems = 8;    // the same in the backward's narrower rows
// Threads per SM that the backward's registers allow (96 a thread, with the next row loaded ahead).
constexpr int kBwdThreadsSM = 640;
// The same with 16 elements (128 registers a thread).
constexpr int kBwdLeanThreads = 512;
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxMin = 1e-30f;

// Sum (or NaN-keeping maximum) over a warp, the same in every lane.
template <bool kMax>
__device__ __forceinline__ float warp_reduce(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = kMax ? max_nan(v, u) : v + u;
    }
    return v;
}

// The same over the threads of a row: a warp, or the CTA (every thread of it calls; each warp combines the
// warps' partials for itself, in one order; 0 is neutral to the sum and to a maximum of magnitudes).  The backward's
// rows wait for this: a loop over the partials and a division by the width took 8192 columns of bf16 from 45 to 67 us.
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v, bool one_warp, float* part) {
    v = warp_reduce<kMax>(v);
    if (one_warp) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_reduce<kMax>(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f);
}

// V weights (16-byte aligned where V > 1), kept in the caches.
template <int V>
__device__ __forceinline__ void load_weights(const float* p, float (&w)[V]) {
    if constexpr (V == 1) {
        w[0] = __ldg(p);
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(p + k));
            w[k] = q.x;
            w[k + 1] = q.y;
            w[k + 2] = q.z;
            w[k + 3] = q.w;
        }
    }
}

template <typename T, typename R, typename O, int V>
__global__ void __launch_bounds__(1024) ssd_add_norm_kernel(AddNormArgs a) {
    constexpr int C = kElems / V;
    __shared__ float part[2][32];
    const bool one_warp = a.rows_per_cta > 1 || blockDim.x == 32;
    const int slot = one_warp ? threadIdx.x >> 5 : 0;
    const int tid = one_warp ? threadIdx.x & 31 : threadIdx.x;
    const int nt = one_warp ? 32 : blockDim.x;
    const int64_t row = (int64_t)blockIdx.x * a.rows_per_cta + slot;
    pdl_wait();
    if (row >= a.rows) return;   // whole warps of a many-row CTA, which has no barrier
    const int W = a.width;
    const size_t base = (size_t)row * W;
    const T* x = static_cast<const T*>(a.x) + base;
    const R* res = a.residual ? static_cast<const R*>(a.residual) + base : nullptr;
    Raw<T, V> xr[C];
    Raw<R, V> rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (tid + c * nt) * V;
        xr[c].zero();
        rr[c].zero();
        if (e < W) {
            xr[c].load(x + e);
            if (res) rr[c].load(res + e);
        }
    }
    float h[C][V];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float r[V];
        xr[c].get(h[c]);
        rr[c].get(r);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            h[c][k] += r[k];
            ss = fmaf(h[c][k], h[c][k], ss);
        }
    }
    ss = row_reduce<false>(ss, one_warp, part[0]);
    const float rstd = 1.f / sqrtf(ss / (float)W + a.eps);
    if (a.rstd && tid == 0) a.rstd[row] = rstd;
    if (a.residual_out) {
        R* ro = static_cast<R*>(a.residual_out) + base;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (tid + c * nt) * V;
            if (e < W) {
                Raw<R, V> q;
                q.set(h[c]);
                q.store(ro + e);
            }
        }
    }
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (tid + c * nt) * V;
        if (e < W) {
            float w[V];
            load_weights(a.weight + e, w);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                h[c][k] = h[c][k] * rstd * w[k];
                amax = max_nan(amax, fabsf(h[c][k]));
            }
        }
    }
    float scale = 1.f, inv = 1.f;
    if constexpr (sizeof(O) == 1) {
        amax = max_nan(row_reduce<true>(amax, one_warp, part[1]), kAmaxMin);
        scale = amax / kE4m3Max;
        if (tid == 0) a.scales[row] = scale;
        inv = 1.f / scale;
        if (inv == 0.f) scale = 0.f;   // an infinite row: the remainders below are then the elements, and change nothing
    }
    O* out = static_cast<O*>(a.out) + base;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (tid + c * nt) * V;
        if (e < W) {
            if constexpr (sizeof(O) == 1) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float q = h[c][k] * inv;
                    h[c][k] = fmaf(fmaf(-q, scale, h[c][k]), inv, q);
                }
            }
            Raw<O, V> q;
            q.set(h[c]);
            q.store(out + e);
        }
    }
}

// E: elements of a row per thread, V of them at a time.  Rows of up to 640 threads of 8 elements, or 512 of 16, have the
// registers to load the next row while the present one is reduced and written; with 16 elements the weights wait in
// shared memory and the residual's gradient is loaded with its own row.
//
// SHIFTED: rows of W elements, W not a multiple of V.  Vectors lie on V-element boundaries of the whole array: a row
// starts `shift` elements into its first one.  Those at its ends hold a neighbour's elements too, which are read with
// them (whatever they are, or are being replaced by: the values are dropped) and never written.  A slot's rows are a
// multiple of 8 apart (or it has one): their shift is one number, and a thread's columns stay its own for dw.
template <typename T, typename R, int V, int E, int THREADS, bool SHIFTED>
__global__ void __launch_bounds__(THREADS) ssd_add_norm_bwd_kernel(AddNormBwdArgs a) {
    constexpr int C = E / V;
    constexpr bool kAhead = E == kBwdElems || THREADS <= kBwdLeanThreads;
    constexpr bool kLean = kAhead && E > kBwdElems;
    __shared__ float part[2][32];
    __shared__ __align__(16) float weights[kLean ? THREADS * E : 1];
    const bool one_warp = a.rows_per_cta > 1 || blockDim.x == 32;
    const int slot = one_warp ? threadIdx.x >> 5 : 0;
    const int tid = one_warp ? threadIdx.x & 31 : threadIdx.x;
    const int nt = one_warp ? 32 : blockDim.x;
    const int W = a.width;
    pdl_trigger();
    pdl_wait();
    const int64_t stride = (int64_t)gridDim.x * a.rows_per_cta;
    int64_t row = (int64_t)blockIdx.x * a.rows_per_cta + slot;
    const int shift = SHIFTED ? (int)((uint64_t)(row * W) % V) : 0;
    // first column of a thread's vector c, and whether all of it lies in the row
    auto column = [&](int c) { return (tid + c * nt) * V - shift; };
    auto whole = [&](int e) { return !SHIFTED || (e >= 0 && e + V <= W); };
    auto in = [&](int e) { return !SHIFTED || (e >= 0 && e < W); };
    auto fetch = [&](auto& v, const auto* p, int64_t row, size_t base, int e) {
        p += base + e;
        if (!SHIFTED || e + V <= W || row + 1 < a.rows) v.load(p);
        else v.load_some(p, W - e);   // the array's last elements
    };
    float dw[C][V], wt[kLean ? 1 : C][V];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = column(c);
        float w[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            dw[c][k] = w[k] = 0.f;
            if (SHIFTED && in(e + k)) w[k] = __ldg(a.weight + e + k);
        }
        if (!SHIFTED && e < W) load_weights(a.weight + e, w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (kLean) weights[(tid + c * nt) * V + k] = w[k];   // read by this thread alone
            else wt[c][k] = w[k];
        }
    }
    struct Row {
        Raw<T, V> d[C];
        Raw<R, V> h[C], s[kLean ? 1 : C];
        float rstd;
    };
    auto load = [&](Row& r, int64_t row) {
        const size_t base = (size_t)row * W;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = column(c);
            r.d[c].zero();
            r.h[c].zero();
            if constexpr (!kLean) r.s[c].zero();
            if (e < W) {
                fetch(r.d[c], static_cast<const T*>(a.dout), row, base, e);
                fetch(r.h[c], static_cast<const R*>(a.h), row, base, e);
                if constexpr (!kLean)
                    if (a.dres) fetch(r.s[c], static_cast<const R*>(a.dres), row, base, e);
            }
        }
        r.rstd = __ldg(a.rstd + row);
    };
    Row cur;
    if (kAhead && row < a.rows) load(cur, row);
    int turn = 0;
    for (; row < a.rows; row += stride) {
        const size_t base = (size_t)row * W;
        Raw<R, V> late[kLean ? C : 1];
        if constexpr (kLean) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = column(c);
                late[c].zero();
                if (a.dres && e < W) fetch(late[c], static_cast<const R*>(a.dres), row, base, e);
            }
        }
        Row next;
        if (kAhead) {
            if (row + stride < a.rows) load(next, row + stride);
        } else {
            load(cur, row);
        }
        float p[C][V], xh[C][V];
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            cur.d[c].get(p[c]);
            cur.h[c].get(xh[c]);
            const int e = column(c);
            if (!whole(e)) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (!in(e + k)) p[c][k] = xh[c][k] = 0.f;
            }
            float w[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if constexpr (kLean) w[k] = weights[(tid + c * nt) * V + k];
                else w[k] = wt[c][k];
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                xh[c][k] *= cur.rstd;
                dw[c][k] = fmaf(p[c][k], xh[c][k], dw[c][k]);
                p[c][k] *= w[k];
                dot = fmaf(p[c][k], xh[c][k], dot);
            }
        }
        // the partials of consecutive rows alternate between two arrays: a row's last
        // reader is past the next row's barrier before a third row writes
        dot = row_reduce<false>(dot, one_warp, part[turn]) * a.inv_width;
        turn ^= 1;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = column(c);
            if (e < W) {
                float s[V];
                if constexpr (kLean) late[c].get(s);
                else cur.s[c].get(s);
#pragma unroll
                for (int k = 0; k < V; ++k) s[k] = fmaf(p[c][k] - xh[c][k] * dot, cur.rstd, s[k]);
                if (a.dx) {
                    T* dx = static_cast<T*>(a.dx) + base;
                    Raw<T, V> q;
                    q.set(s);
                    if (whole(e)) q.store(dx + e);
                    else q.store_within(dx, e, W);
                }
                if (a.dres_out) {
                    R* dr = static_cast<R*>(a.dres_out) + base;
                    Raw<R, V> q;
                    q.set(s);
                    if (whole(e)) q.store(dr + e);
                    else q.store_within(dr, e, W);
                }
            }
        }
        if (kAhead) cur = next;
    }
    float* share = a.shares + ((size_t)blockIdx.x * a.rows_per_cta + slot) * W;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = column(c);
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (e < W && in(e + k)) share[e + k] = dw[c][k];
    }
}

// dw[e] = sum over the shares: COLS columns (16 or 32) per CTA, the shares dealt to its 1024 / COLS rows of threads, whose
// sums are added in their order.
template <int COLS>
__global__ void __launch_bounds__(1024) ssd_add_norm_bwd_reduce(const float* shares, int nshares, int W, float* dw) {
    __shared__ float part[32][COLS + 1];
    const int lane = threadIdx.x % COLS, w = threadIdx.x / COLS;
    const int e = blockIdx.x * COLS + lane;
    float s = 0.f;
    pdl_trigger();
    pdl_wait();   // launched while the shares are still being summed
    if (e < W) {
#pragma unroll 4
        for (int k = w; k < nshares; k += 1024 / COLS) s += shares[(size_t)k * W + e];
    }
    if (COLS == 16) s += __shfl_xor_sync(0xffffffffu, s, 16);   // the warp's two rows
    if ((threadIdx.x & 31) < COLS) part[threadIdx.x >> 5][lane] = s;
    __syncthreads();
    if (threadIdx.x < COLS && e < W) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) t += part[k][lane];
        dw[e] = t;
    }
}

struct RowShape {
    int threads, rows_per_cta;
};

RowShape row_shape(int width, int64_t rows, int elems) {
    RowShape s;
    if (width <= 32 * elems) {
        s.rows_per_cta = rows < 4 ? (int)rows : 4;
        s.threads = 32 * s.rows_per_cta;
    } else {
        s.rows_per_cta = 1;
        s.threads = ((width + elems - 1) / elems + 31) / 32 * 32;
    }
    return s;
}

// Elements that the backward's vectors of a row span: rows of other than whole vectors may reach into one more.
int bwd_span(int width) { return width % 8 == 0 ? width : width + 7; }

// Elements per thread of the backward: 8 where 640 threads of 8 span a row, else 16; lean: 16 beyond 1280 columns already.
int bwd_elems(int width, bool lean) {
    const int span = bwd_span(width);
    return span > kBwdThreadsSM * kBwdElems || (lean && span > 1280) ? kElems : kBwdElems;
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, typename R, typename O>
cudaError_t launch_fwd_typed(const AddNormArgs& a, int threads, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.width % V == 0 && on16(a.weight) && on16(a.x) && on16(a.residual) && on16(a.out) && on16(a.residual_out);
    const unsigned grid = (unsigned)((a.rows + a.rows_per_cta - 1) / a.rows_per_cta);
    return launch_kernel(vec ? ssd_add_norm_kernel<T, R, O, V> : ssd_add_norm_kernel<T, R, O, 1>, grid, (unsigned)threads, 0, st, true, a);
}

template <typename T, typename R>
cudaError_t launch_fwd_res(const AddNormArgs& a, int threads, cudaStream_t st) {
    if (a.out_dtype == SSD_E4M3) return launch_fwd_typed<T, R, e4m3_t>(a, threads, st);
    return launch_fwd_typed<T, R, T>(a, threads, st);
}

// Row slots of the backward's grid: as many as fill the SMs, so that each slot's
// dw share sums many rows and the shares stay a few percent of the traffic.
// Slots with several rows have 152 n CTAs' rows between them, a multiple of 8.
static_assert(kAddNormSMs % 8 == 0, "a slot's rows keep their shift");
int64_t bwd_slots(int64_t rows, int width, bool lean, int* rows_per_cta, int* threads, int64_t* grid) {
    const int elems = bwd_elems(width, lean);
    const RowShape s = row_shape(bwd_span(width), rows, elems);
    const int room = elems == kBwdElems ? kBwdThreadsSM : kBwdLeanThreads;
    const int per_sm = room / s.threads > 0 ? room / s.threads : 1;
    int64_t g = (rows + s.rows_per_cta - 1) / s.rows_per_cta;
    const int64_t most = (int64_t)kAddNormSMs * per_sm;
    if (g > most) g = most;
    *rows_per_cta = s.rows_per_cta;
    *threads = s.threads;
    *grid = g;
    return g * s.rows_per_cta;
}

// 16-byte vectors where every array starts on 16 bytes and rows hold one at least, elements otherwise.  33.5 M elements,
// us by the rule and by the other side of it (fp32 residual unless said):
//   lean, bf16 beyond 1280 columns   2048 columns 86.7 (8 elements 87.6), 2560 85.9 (84.0), 4096 87.9 (91.1); bf16 residual 2048
//                                    49.9 (59.9), 2560 50.9 (52.0), 4096 52.0 (58.0); no residual 2048 40.9 (56.4), 4096 41.7 (52.6)
//   not lean, bf16 up to there       1024 columns 83.1 (16 elements 130.9), 1280 82.5 (101.2); bf16 residual 1024 52.0 (72.7), 1280
//                                    51.1 (73.9); no residual 512 46.6 (40.1), 1024 47.1 (57.4), 1280 44.8 (57.8)
//   where the other side is faster   1536 columns, whose rows are 96 threads of 16: 96.4 (84.3), 66.1 (55.5), 54.2 (51.6); 5120, one CTA an
//                                    SM either way: 87.4 (87.6), 65.1 (53.1), 49.9 (47.7)
//   not lean, fp32                   5120 columns 85.4 (16 elements 97.2; it spills)
//   not lean, bf16 shifted           2049 columns 99 (112; it spills), 4001 102 (107); bf16 residual lean, 4001 53 (62)
//   rows beyond 5120 columns         8192 columns 91.6, fp32 83.7, bf16 residual 45 (1024 threads of 8, without the
//                                    next row ahead: 119, 106)
//   shifted vectors                  6001 columns 117, fp32 116 (elements 148, 139)
template <typename T, typename R>
cudaError_t launch_bwd_typed(AddNormBwdArgs& a, int64_t* nshares, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool shifted = a.width % V != 0;
    const bool vec = a.width >= V && bwd_span(a.width) <= 1024 * kElems && on16(a.dout) && on16(a.h) && on16(a.dres) &&
                     on16(a.dx) && on16(a.dres_out) && (shifted || on16(a.weight));
    const bool lean = vec && sizeof(T) == 2 && (!shifted || sizeof(R) == 2);
    int threads;
    int64_t grid;
    *nshares = bwd_slots(a.rows, a.width, lean, &a.rows_per_cta, &threads, &grid);
    void (*kern)(AddNormBwdArgs);
    if (bwd_elems(a.width, lean) == kBwdElems)
        kern = !vec      ? ssd_add_norm_bwd_kernel<T, R, 1, kBwdElems, kBwdThreadsSM, false>
               : shifted ? ssd_add_norm_bwd_kernel<T, R, V, kBwdElems, kBwdThreadsSM, true>
                         : ssd_add_norm_bwd_kernel<T, R, V, kBwdElems, kBwdThreadsSM, false>;
    else if (vec && threads <= kBwdLeanThreads)
        kern = shifted ? ssd_add_norm_bwd_kernel<T, R, V, kElems, kBwdLeanThreads, true>
                       : ssd_add_norm_bwd_kernel<T, R, V, kElems, kBwdLeanThreads, false>;
    else
        kern = !vec      ? ssd_add_norm_bwd_kernel<T, R, 1, kElems, 1024, false>
               : shifted ? ssd_add_norm_bwd_kernel<T, R, V, kElems, 1024, true>
                         : ssd_add_norm_bwd_kernel<T, R, V, kElems, 1024, false>;
    return launch_kernel(kern, (unsigned)grid, threads < 1024 ? threads : 1024, 0, st, true, a);
}

}  // namespace

cudaError_t launch_add_norm(const AddNormArgs& args, cudaStream_t st) {
    AddNormArgs a = args;
    const RowShape s = row_shape(a.width, a.rows, kElems);
    a.rows_per_cta = s.rows_per_cta;
    if (a.dtype == SSD_BF16)
        return a.residual_dtype == SSD_F32 ? launch_fwd_res<bf16_t, float>(a, s.threads, st)
                                           : launch_fwd_res<bf16_t, bf16_t>(a, s.threads, st);
    return launch_fwd_res<float, float>(a, s.threads, st);
}

// Enough for either shape: which one a call takes depends on its addresses too.
int64_t add_norm_bwd_shares(int64_t rows, int width) {
    int rpc, threads;
    int64_t grid;
    const int64_t n = bwd_slots(rows, width, false, &rpc, &threads, &grid);
    const int64_t m = bwd_slots(rows, width, true, &rpc, &threads, &grid);
    return n > m ? n : m;
}

cudaError_t launch_add_norm_bwd(const AddNormBwdArgs& args, cudaStream_t st) {
    AddNormBwdArgs a = args;
    a.inv_width = 1.f / (float)a.width;
    int64_t nshares;
    cudaError_t e;
    if (a.dtype == SSD_BF16)
        e = a.residual_dtype == SSD_F32 ? launch_bwd_typed<bf16_t, float>(a, &nshares, st)
                                        : launch_bwd_typed<bf16_t, bf16_t>(a, &nshares, st);
    else
        e = launch_bwd_typed<float, float>(a, &nshares, st);
    if (e != cudaSuccess) return e;
    // 16 columns a CTA while all CTAs run at once (20000 x 256 in a graph 17.2 us, with 32 18.6; 4096 x 8192 94 and 89)
    const int cols = a.width <= 16 * 2 * kAddNormSMs ? 16 : 32;
    return launch_kernel(cols == 16 ? ssd_add_norm_bwd_reduce<16> : ssd_add_norm_bwd_reduce<32>, (unsigned)((a.width + cols - 1) / cols),
                         1024, 0, st, true, (const float*)a.shares, (int)nshares, a.width, a.dweight);
}

}  // namespace ssd
