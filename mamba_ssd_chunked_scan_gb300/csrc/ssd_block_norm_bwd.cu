// Gradients of the norm after a block (ssd_block_norm_kernel's formula) and of the gate and grouped norm after the scan:
//   ssd_block_norm_bwd_kernel   p2 = next_weight dout, hh = h rstd2:  dh = dres + rstd2 (p2 - hh mean(p2 hh))
//                               p1 = scale dh weight,  uh = u rstd1:  du = rstd1 (p1 - uh mean(p1 uh))
//                               dx = du silu(gate),  dgate = du x s (1 + gate (1 - s)),  s = 1 / (1 + e^-gate)
//                               and each row slot's shares of  dweight = sum scale dh uh,  dnext_weight = sum dout hh
//   (without a residual: scale dh is dout itself)
//
// u and both rstd are recomputed from x, gate and h, which may be 8-bit rows.  A grid as large as the GPU holds at
// once walks the rows, so that the shares stay few; ssd_share_sum adds them in a fixed order.
//
// Up to five operands a row are too many to keep the next row's in registers, and HBM wants some 50 KB in flight per
// SM.  So each thread copies its own vectors of the rows to come into slots of its own in shared memory (cp.async), up to
// three rows ahead: no barrier and no register holds them.  The weights lie there too.  Where rows are no whole vectors, the vectors
// are those of the whole array (see SHIFTED).
#include <atomic>

#include "ssd_kernels.h"
#include "ssd_rows.cuh"

namespace ssd {
namespace {

constexpr int kMaxStages = 4;
constexpr int kWideElems = 16, kNarrowElems = 8;   // elements of a row per thread
constexpr int kSmemSM = 228 * 1024, kSmemCta = 227 * 1024;
constexpr int kSmemOwn = 2048;                     // a CTA's static shared memory and what the system takes

// Copies of 16, 8 or 4 bytes, of which the first `n` are read and the others 0.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int n) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most the newest `n` groups of copies are under way.
__device__ __forceinline__ void copies_wait(int n) {
    if (n == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A row's operands, the order of their slots in a stage.
enum Operand { kDout, kX, kGate, kH, kDres, kOperands };

// E elements of a row per thread, V of them together: V > 1, 16 bytes of T through shared memory; V = 1, anything,
// straight from memory.
//
// SHIFTED: rows of n elements, n not a multiple of V.  Vectors lie on V-element boundaries of the whole array: a row
// starts `shift` elements into its first one.  Those at its ends hold a neighbour's elements too, which are read with them
// (and dropped) and never written.  A slot's rows are a multiple of 8 apart (or it has one): their shift is one number, and a
// thread's columns stay its own for the weights' gradients.
template <typename T, typename R, int V, int E, int THREADS, bool SHIFTED, bool GATE, bool RES>
__global__ void __launch_bounds__(THREADS) ssd_block_norm_bwd_kernel(BlockNormBwdArgs a) {
    constexpr int C = E / V;
    constexpr bool kRing = V > 1;
    __shared__ float4 part[2][32];
    extern __shared__ __align__(16) unsigned char ring[];
    const bool one_warp = a.slots_per_cta > 1 || blockDim.x == 32;
    const int slot = one_warp ? threadIdx.x >> 5 : 0;
    const int tid = one_warp ? threadIdx.x & 31 : threadIdx.x;
    const int nt = one_warp ? 32 : blockDim.x;
    const int id = blockIdx.x * a.slots_per_cta + slot;
    pdl_trigger();
    pdl_wait();
    if (id >= a.slots) return;   // whole warps of a many-slot CTA, which has no barrier
    const int n = a.size;
    const int line = id / a.groups, group = id - line * a.groups, first = group * n;   // the slot's first row, its group's first column
    const int64_t step = a.slots / a.groups;
    const bool next = RES && a.dout;
    const int shift = SHIFTED ? (int)((uint64_t)((int64_t)line * a.groups + group) * n % V) : 0;
    // first column of a thread's vector c, and whether all of it lies in the row
    auto column = [&](int c) { return (tid + c * nt) * V - shift; };
    auto whole = [&](int e) { return !SHIFTED || (e >= 0 && e + V <= n); };
    auto write = [&](auto* row, int e, const auto& v) {
        Raw<typename std::remove_pointer<decltype(row)>::type, V> q;
        q.set(v);
        if (whole(e)) q.store(row + e);
        else q.store_within(row, e, n);
    };
    // the slot's shared memory: its weights, then its stages
    unsigned char* const mine = ring + (size_t)slot * a.slot_bytes;
    float4* const wslots = reinterpret_cast<float4*>(mine);
    unsigned char* const stages = mine + a.weight_bytes;
    if constexpr (kRing) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = column(c);
            if (e >= n) continue;
#pragma unroll
            for (int which = 0; which < (RES ? 2 : 1); ++which) {
                float w[V];
                const float* p = which ? a.next_weight : a.weight + first;
                if (!p) continue;
                row_weights<V, SHIFTED>(p, e, n, w);
#pragma unroll
                for (int q = 0; q < V / 4; ++q)
                    wslots[((which * C + c) * (V / 4) + q) * nt + tid] = make_float4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
            }
        }
    }
    auto weights = [&](int which, int c, float (&w)[V]) {
        if constexpr (kRing) {
#pragma unroll
            for (int q = 0; q < V / 4; ++q) {
                const float4 f = wslots[((which * C + c) * (V / 4) + q) * nt + tid];
                w[4 * q] = f.x;
                w[4 * q + 1] = f.y;
                w[4 * q + 2] = f.z;
                w[4 * q + 3] = f.w;
            }
        } else {
            row_weights<1, false>(which ? a.next_weight : a.weight + first, column(c), n, w);
        }
    };
    // Ask for a row's operands into a stage's slots.
    auto ask = [&](int64_t row, int stage) {
        if constexpr (kRing) {
            const int64_t unit = row * a.groups + group;
            const size_t base = (size_t)unit * n, gbase = GATE ? (size_t)row * a.gate_stride + first : 0;
            const int64_t left = SHIFTED ? ((int64_t)a.rows * a.groups - unit) * n : 0;   // elements to the arrays' end
            unsigned char* const to = stages + (size_t)stage * a.stage_bytes;
            auto vector = [&](auto* type, const void* p, const float* scales, int operand, size_t at, int c, int count) {
                constexpr int kSize = sizeof(*type);
                const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to + a.offset[operand]);
                if (scales) {
                    copy_async<V>(dst + (c * nt + tid) * V, static_cast<const e4m3_t*>(p) + at, count);
                } else {
#pragma unroll
                    for (int h = 0; h < kSize * V / 16; ++h) {
                        const int bytes = count * kSize - 16 * h;
                        const int some = bytes < 0 ? 0 : bytes < 16 ? bytes : 16;
                        copy_async<16>(dst + ((c * (kSize * V / 16) + h) * nt + tid) * 16,
                                       static_cast<const unsigned char*>(p) + at * kSize + (some > 0 ? 16 * h : 0), some);
                    }
                }
            };
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = column(c);
                if (e >= n) continue;
                const int count = SHIFTED && left - e < V ? (int)(left - e) : V;
                const size_t at = base + e;
                if (!RES || next) vector((T*)nullptr, a.dout, nullptr, kDout, at, c, count);
                vector((T*)nullptr, a.x, a.x_scales, kX, at, c, count);
                if (GATE) vector((T*)nullptr, a.gate, a.gate_scales, kGate, gbase + e, c, count);
                if (next) vector((R*)nullptr, a.h, a.h_scales, kH, at, c, count);
                if (RES) vector((R*)nullptr, a.dres, nullptr, kDres, at, c, count);
            }
            auto scale = [&](const float* scales, int operand) {
                if (scales) copy_async<4>((uint32_t)__cvta_generic_to_shared(to + a.scale_offset[operand]) + 4 * tid, scales + unit, 4);
            };
            scale(a.x_scales, kX);
            if (GATE) scale(a.gate_scales, kGate);
            if (next) scale(a.h_scales, kH);
            copies_commit();
        }
    };
    float dw[C][V], dn[RES ? C : 1][V];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            dw[c][k] = 0.f;
            if (RES) dn[c][k] = 0.f;
        }
    int64_t ahead = line;   // the next row to ask for, and its stage
    int fill = 0;
    if constexpr (kRing) {
        for (; fill < a.stages - 1; ++fill, ahead += step) {
            if (ahead < a.rows) ask(ahead, fill);
            else copies_commit();
        }
    }
    int turn = 0, stage = 0;
    for (int64_t row = line; row < a.rows; row += step) {
        const int64_t unit = row * a.groups + group;
        const size_t base = (size_t)unit * n, gbase = GATE ? (size_t)row * a.gate_stride + first : 0;
        unsigned char* const from = stages + (size_t)stage * a.stage_bytes;
        if constexpr (kRing) {
            if (ahead < a.rows) ask(ahead, fill);
            else copies_commit();
            ahead += step;
            if (++fill == a.stages) fill = 0;
            if (++stage == a.stages) stage = 0;
            copies_wait(a.stages - 1);
        }
        auto row_scale = [&](const float* scales, int operand) {
            if (!scales) return 1.f;
            if constexpr (kRing) return *reinterpret_cast<const float*>(from + a.scale_offset[operand] + 4 * tid);
            else return __ldg(scales + unit);
        };
        const float xs = row_scale(a.x_scales, kX), gs = GATE ? row_scale(a.gate_scales, kGate) : 1.f, hs = next ? row_scale(a.h_scales, kH) : 1.f;
        // A thread's vector c of an operand: of type T or R, or 8-bit codes times the row's scale.
        auto take = [&](auto* type, const void* p, const float* scales, float s, int operand, size_t at, int c, float (&v)[V]) {
            typedef typename std::remove_pointer<decltype(type)>::type K;
            if (scales) {
                Raw<e4m3_t, V> q;
                if constexpr (kRing) q.w = *reinterpret_cast<const typename Raw<e4m3_t, V>::W*>(from + a.offset[operand] + (c * nt + tid) * V);
                else q.load(static_cast<const e4m3_t*>(p) + at);
                from_codes(q, v);
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] *= s;
            } else {
                Raw<K, V> q;
                if constexpr (kRing) {
                    constexpr int H = sizeof(K) * V / 16;
                    const uint4* slots = reinterpret_cast<const uint4*>(from + a.offset[operand]) + c * H * nt + tid;
                    if constexpr (H == 2) {
                        q.w.lo = slots[0];
                        q.w.hi = slots[nt];
                    } else {
                        q.w = slots[0];
                    }
                } else {
                    q.load(static_cast<const K*>(p) + at);
                }
                q.get(v);
            }
            if constexpr (SHIFTED) {
                const int e = column(c);
                if (!whole(e)) {
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (e + k < 0 || e + k >= n) v[k] = 0.f;
                }
            }
        };
        // u (kept), and what the first means need
        float u[C][V], sg[GATE ? C : 1][V], g1[C][V];   // g1: the gradient of u rstd1 weight
        RowSums s = {0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = column(c);
#pragma unroll
            for (int k = 0; k < V; ++k) u[c][k] = g1[c][k] = 0.f;
            if (e >= n) continue;
            take((T*)nullptr, a.x, a.x_scales, xs, kX, base + e, c, u[c]);
            if (GATE) {
                float g[V];
                take((T*)nullptr, a.gate, a.gate_scales, gs, kGate, gbase + e, c, g);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    sg[c][k] = sigmoid<T>(g[k]);
                    u[c][k] *= g[k] * sg[c][k];
                }
            }
#pragma unroll
            for (int k = 0; k < V; ++k) s.a = fmaf(u[c][k], u[c][k], s.a);
            float w[V];
            if constexpr (RES) {
                if (next) {
                    float h[V], d[V];
                    take((R*)nullptr, a.h, a.h_scales, hs, kH, base + e, c, h);
                    take((T*)nullptr, a.dout, nullptr, 1.f, kDout, base + e, c, d);
                    weights(1, c, w);
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        s.b = fmaf(h[k], h[k], s.b);
                        s.c = fmaf(d[k] * w[k], h[k], s.c);
                    }
                }
            } else {
                take((T*)nullptr, a.dout, nullptr, 1.f, kDout, base + e, c, g1[c]);
                weights(0, c, w);
#pragma unroll
                for (int k = 0; k < V; ++k) s.b = fmaf(g1[c][k] * w[k], u[c][k], s.b);
            }
        }
        row_sums<RES ? 3 : 2>(s, one_warp, part[turn]);
        turn ^= 1;
        const float rstd = 1.f / sqrtf(s.a * a.inv_size + a.eps);
        if constexpr (RES) {
            const float rstd2 = next ? 1.f / sqrtf(s.b * a.inv_size + a.eps) : 0.f;
            const float mean2 = s.c * rstd2 * rstd2 * a.inv_size;   // h times it is hh mean(p2 hh)
            RowSums t = {0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = column(c);
                if (e >= n) continue;
                float dh[V], w[V];
                take((R*)nullptr, a.dres, nullptr, 1.f, kDres, base + e, c, dh);
                if (next) {
                    float h[V], d[V];
                    take((R*)nullptr, a.h, a.h_scales, hs, kH, base + e, c, h);
                    take((T*)nullptr, a.dout, nullptr, 1.f, kDout, base + e, c, d);
                    weights(1, c, w);
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        dh[k] = fmaf(rstd2, fmaf(d[k], w[k], -h[k] * mean2), dh[k]);
                        dn[c][k] = fmaf(d[k], h[k] * rstd2, dn[c][k]);
                    }
                }
                write(static_cast<R*>(a.dres_out) + base, e, dh);
                weights(0, c, w);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    g1[c][k] = a.scale * dh[k];
                    t.a = fmaf(g1[c][k] * w[k], u[c][k], t.a);
                }
            }
            row_sums<1>(t, one_warp, part[turn]);
            turn ^= 1;
            s.b = t.a;
        }
        const float mean1 = s.b * rstd * rstd * a.inv_size;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = column(c);
            if (e >= n) continue;
            float w[V], du[V];
            weights(0, c, w);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                du[k] = rstd * fmaf(g1[c][k], w[k], -u[c][k] * mean1);
                dw[c][k] = fmaf(g1[c][k], u[c][k] * rstd, dw[c][k]);
            }
            if (!RES && a.out) {
                float o[V];
#pragma unroll
                for (int k = 0; k < V; ++k) o[k] = u[c][k] * rstd * w[k];
                write(static_cast<T*>(a.out) + base, e, o);
            }
            if (GATE) {
                float x[V], g[V], dg[V];
                take((T*)nullptr, a.x, a.x_scales, xs, kX, base + e, c, x);
                take((T*)nullptr, a.gate, a.gate_scales, gs, kGate, gbase + e, c, g);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float b = g[k] * sg[c][k];
                    dg[k] = du[k] * x[k] * fmaf(sg[c][k], 1.f - b, b);   // s + gate s (1 - s)
                    du[k] *= b;
                }
                write(static_cast<T*>(a.dgate) + (size_t)row * a.dgate_stride + first, e, dg);
            }
            write(static_cast<T*>(a.dx) + base, e, du);
        }
    }
    const int width = n * a.groups, columns = RES && a.next_weight ? 2 * width : width;
    float* share = a.shares + (size_t)line * columns + first;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = column(c);
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (e + k >= 0 && e + k < n) {
                share[e + k] = dw[c][k];
                if (RES && a.next_weight) share[width + e + k] = dn[c][k];
            }
    }
}

// How a call's rows are spread: threads of a CTA, its slots, and all slots (`lines` rows at a time, each of its groups).
struct Plan {
    int threads, slots_per_cta, slots, grid;
};

// Threads per SM that the registers of E elements a thread allow.
constexpr int threads_sm(int elems) { return elems == kNarrowElems ? 640 : 512; }

// Elements per thread where vectors are taken: 8 while that makes at most 320 threads.
int vector_elems(int span) { return span <= 320 * kNarrowElems ? kNarrowElems : kWideElems; }

Plan plan(int64_t rows, int span, int groups, int elems, int per_sm) {
    Plan p;
    int cta_slots = 1;
    p.threads = ((span + elems - 1) / elems + 31) / 32 * 32;
    if (p.threads == 32) cta_slots = 4;
    int64_t lines = (int64_t)kAddNormSMs * per_sm * cta_slots / groups / 8 * 8;
    if (lines < 8) lines = 8;
    if (lines > rows) lines = rows;
    p.slots = (int)lines * groups;
    p.slots_per_cta = p.slots < cta_slots ? p.slots : cta_slots;
    p.threads *= p.slots_per_cta;
    p.grid = (p.slots + p.slots_per_cta - 1) / p.slots_per_cta;
    return p;
}
// CTAs that an SM's registers hold.
int ctas_sm(int span, int elems) {
    int threads = ((span + elems - 1) / elems + 31) / 32 * 32;
    if (threads == 32) threads = 128;
    return threads_sm(elems) / threads > 0 ? threads_sm(elems) / threads : 1;
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }
int vector_span(int size) { return size % 8 == 0 ? size : size + 7; }

template <typename T, typename R, int V, int E, bool SHIFTED, bool GATE, bool RES>
cudaError_t launch_one(const BlockNormBwdArgs& a, const Plan& p, size_t smem, cudaStream_t st) {
    constexpr int kThreads = V == 1 ? 512 : threads_sm(E);
    auto kern = ssd_block_norm_bwd_kernel<T, R, V, E, kThreads, SHIFTED, GATE, RES>;
    static std::atomic<uint8_t> ready[kMaxDevices];
    if (V > 1) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
        if (!ready[dev].load(std::memory_order_acquire)) {
            if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemCta - kSmemOwn)) != cudaSuccess ||
                (e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
                return e;
            ready[dev].store(1, std::memory_order_release);
        }
    }
    return launch_kernel(kern, (unsigned)p.grid, (unsigned)p.threads, smem, st, true, a);
}

template <typename T, typename R, bool GATE, bool RES>
cudaError_t launch_typed(BlockNormBwdArgs& a, int* lines, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    auto aligned = [&](const void* q, bool packed) { return packed ? ((uintptr_t)q % V) == 0 : on16(q); };
    const bool shifted = a.size % V != 0;
    const int span = vector_span(a.size), width = a.size * a.groups;
    const bool vec = a.size >= V && span <= 512 * kWideElems && aligned(a.x, a.x_scales) && aligned(a.h, a.h_scales) && on16(a.dout) &&
                     on16(a.dres) && on16(a.dres_out) && on16(a.dx) && on16(a.out) &&
                     (shifted || (on16(a.weight) && on16(a.next_weight))) &&
                     (!GATE || (aligned(a.gate, a.gate_scales) && on16(a.dgate) &&
                                (shifted ? a.gate_stride == width && a.dgate_stride == width : a.gate_stride % V == 0 && a.dgate_stride % V == 0)));
    if (!vec) {
        const Plan p = plan(a.rows, a.size, a.groups, kWideElems, ctas_sm(a.size, kWideElems));
        a.slots = p.slots;
        a.slots_per_cta = p.slots_per_cta;
        *lines = p.slots / a.groups;
        return launch_one<T, R, 1, kWideElems, false, GATE, RES>(a, p, 0, st);
    }
    // a stage: the operands' vectors, and a word a thread for each scale
    const int elems = vector_elems(span);
    const int cta = ((span + elems - 1) / elems + 31) / 32 * 32;   // a slot's threads
    const bool next = RES && a.dout;
    int bytes = 0;
    auto put = [&](int operand, bool there, bool packed, int size) {
        a.offset[operand] = bytes;
        if (there) bytes += cta * elems * (packed ? 1 : size);
    };
    put(kDout, !RES || next, false, sizeof(T));
    put(kX, true, a.x_scales, sizeof(T));
    put(kGate, GATE, a.gate_scales, sizeof(T));
    put(kH, next, a.h_scales, sizeof(R));
    put(kDres, RES, false, sizeof(R));
    auto put_scale = [&](int operand, bool there) {
        a.scale_offset[operand] = bytes;
        if (there) bytes += 4 * cta;
    };
    put_scale(kX, a.x_scales);
    put_scale(kGate, GATE && a.gate_scales);
    put_scale(kH, next && a.h_scales);
    a.stage_bytes = bytes;
    a.weight_bytes = cta * elems * 4 * (next ? 2 : 1);
    const int cta_slots = cta == 32 ? 4 : 1;
    int per_sm = ctas_sm(span, elems);
    for (;; --per_sm) {
        const int room = (kSmemSM / per_sm < kSmemCta + 1024 ? kSmemSM / per_sm : kSmemCta + 1024) - 1024 - kSmemOwn;
        a.stages = (room / cta_slots - a.weight_bytes) / a.stage_bytes;
        if (a.stages >= 2 || per_sm == 1) break;
    }
    if (a.stages < 1) return cudaErrorInvalidValue;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    a.slot_bytes = a.weight_bytes + a.stages * a.stage_bytes;
    const Plan p = plan(a.rows, span, a.groups, elems, per_sm);
    a.slots = p.slots;
    a.slots_per_cta = p.slots_per_cta;
    *lines = p.slots / a.groups;
    const size_t smem = (size_t)a.slot_bytes * p.slots_per_cta;
    if (elems == kNarrowElems)
        return shifted ? launch_one<T, R, V, kNarrowElems, true, GATE, RES>(a, p, smem, st) : launch_one<T, R, V, kNarrowElems, false, GATE, RES>(a, p, smem, st);
    return shifted ? launch_one<T, R, V, kWideElems, true, GATE, RES>(a, p, smem, st) : launch_one<T, R, V, kWideElems, false, GATE, RES>(a, p, smem, st);
}

}  // namespace

// Enough for every shape: which one a call takes depends on its addresses and types too.
int64_t block_norm_bwd_lines(int64_t rows, int size, int groups) {
    const int span = vector_span(size), elems = vector_elems(span);
    const Plan p = plan(rows, span, groups, elems, ctas_sm(span, elems)), q = plan(rows, size, groups, kWideElems, ctas_sm(size, kWideElems));
    return (p.slots > q.slots ? p.slots : q.slots) / groups;
}

cudaError_t launch_block_norm_bwd(const BlockNormBwdArgs& args, cudaStream_t st) {
    BlockNormBwdArgs a = args;
    a.inv_size = 1.f / (float)a.size;
    int lines = 0;
    cudaError_t e;
    if (!a.dres)
        e = a.dtype == SSD_BF16 ? launch_typed<bf16_t, bf16_t, true, false>(a, &lines, st) : launch_typed<float, float, true, false>(a, &lines, st);
    else if (a.dtype == SSD_F32)
        e = a.gate ? launch_typed<float, float, true, true>(a, &lines, st) : launch_typed<float, float, false, true>(a, &lines, st);
    else if (a.residual_dtype == SSD_F32)
        e = a.gate ? launch_typed<bf16_t, float, true, true>(a, &lines, st) : launch_typed<bf16_t, float, false, true>(a, &lines, st);
    else
        e = a.gate ? launch_typed<bf16_t, bf16_t, true, true>(a, &lines, st) : launch_typed<bf16_t, bf16_t, false, true>(a, &lines, st);
    if (e != cudaSuccess) return e;
    const int width = a.size * a.groups;
    return launch_share_sum(a.shares, lines, width, a.next_weight ? 2 * width : width, a.dweight, a.dnext_weight, st);
}

}  // namespace ssd
