// The norm after a block, with the block's gate, the scaled residual addition and the next block's norm, in one pass:
//   ssd_block_norm_kernel   u = x silu(gate)  (or x)
//                           n = u rstd1 weight,                     rstd1 = 1 / sqrt(mean(u^2) + eps)
//                           h = residual + scale n                  (or, without a residual, out = n)
//                           out = h rstd2 next_weight,              rstd2 = 1 / sqrt(mean(h^2) + eps)
// and x and gate as 8-bit rows, for the backward pass.
//
// A row is read once and written once; h is normalised as it was summed, before its rounding to the residual's type.  A slot
// (a CTA, or lanes of a warp for groups of up to 256 columns) takes some rows one after another, the next ones on their
// way through shared memory (ssd_ring.cuh) while one is worked on: a row a CTA, from registers, left HBM idle between a row's
// loads and its stores (16384 x 5120 with its checkpoint 148 us).  Slots take few rows, so that SMs share the work as
// they finish.  Where no vectors fit, single elements go through registers.
//
// HBM bounds it: gate and norm of 16384 x 5120 bf16 with its checkpoint 104 us, 95 % of the copy's rate; norm after a gated block of
// 16384 x 2560, bf16 beside an fp32 residual, with its checkpoint 107 us, 93 %; 65536 x 1024 without gate and checkpoint 119 us, all of it.
#include <atomic>

#include "ssd_kernels.h"
#include "ssd_ring.cuh"

namespace ssd {
namespace {

// Threads per SM that the registers of E elements a thread allow.
constexpr int fwd_threads_sm(int elems) { return elems == kNarrowElems ? 960 : 640; }

// A warp's record of one row, as in ssd_block_norm_bwd.cuh.
template <typename T, typename R, int E, bool GATE, bool RES>
struct Record {
    static constexpr int t = E * (int)sizeof(T), r = RES ? E * (int)sizeof(R) : 0;
    static constexpr int res = 0, x = r, gate = x + t, bytes = gate + (GATE ? t : 0);
    static constexpr int weight = E * 4, weights = (RES ? 2 : 1) * weight;
};

// Vector c of a row (from column e, the first of its codes at `row`) times inv as codes; `bad`: some element of the row is infinite or NaN.
template <int V, bool SHIFTED>
__device__ __forceinline__ void put_codes(e4m3_t* row, uint32_t off, int e, int n, Two (&v)[V / 2], float inv, bool bad) {
    if (bad) {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) v[k] = two(nan_unless_finite(low(v[k])), nan_unless_finite(high(v[k])));
    }
#pragma unroll
    for (int k = 0; k < V / 2; ++k) v[k] = v[k] * both(inv);
    put<e4m3_t, V, SHIFTED>(reinterpret_cast<unsigned char*>(row), off, e, n, 0u, v);
}

template <typename T, typename R, int E, int LANES, bool SHIFTED, bool GATE, bool RES>
__global__ void __launch_bounds__(fwd_threads_sm(E)) ssd_block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
    typedef Record<T, R, E, GATE, RES> Rec;
    constexpr int V = 16 / (int)sizeof(T), C = E / V, P = V / 2;
    constexpr int kX = 32 * Rec::x, kZ = 32 * Rec::gate, kR = 32 * Rec::res, kStage = 32 * Rec::bytes;
    constexpr bool kCta = LANES == 0;
    constexpr bool kPairs = RES && sizeof(R) > sizeof(T);   // lanes copy for their neighbours
    __shared__ RowPart part[2];
    __shared__ uint32_t tops[2][32];
    extern __shared__ __align__(16) unsigned char ring[];
    const uint32_t mask = row_mask<LANES>();
    const int tid = kCta ? threadIdx.x : threadIdx.x % (kCta ? 32 : LANES), nt = kCta ? blockDim.x : LANES;
    const uint32_t id = kCta ? blockIdx.x : blockIdx.x * a.units_per_cta + threadIdx.x / (kCta ? 32 : LANES);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    if (id >= a.slots) return;   // all of a row's lanes
    const int n = a.size;
    const uint32_t line = a.groups == 1 ? id : id / (uint32_t)a.groups, units = (uint32_t)a.units;
    const int group = (int)(id - line * a.groups), first = group * n;   // the group's first column
    const int shift = SHIFTED ? (int)((uint64_t)id * n & (V - 1)) : 0;
    const int e0 = tid * V - shift, span = nt * V;
    unsigned char* const wrec = ring + warp * (32 * Rec::weights + a.stages * kStage);
    unsigned char* const rec0 = wrec + 32 * Rec::weights;
    // elements from an array's start to vector 0 of thread 0, and between the slot's rows; unit: the row and group at hand
    const int64_t far = (int64_t)a.slots * n, gate_far = (int64_t)(a.slots / a.groups) * a.gate_stride;
    int64_t at = (int64_t)id * n - shift;
    auto in = [](const void* p, int64_t elems, int size) { return static_cast<const unsigned char*>(p) + elems * size; };
    const unsigned char *p_x = in(a.x, at, sizeof(T)), *p_gate = in(a.gate, (int64_t)line * a.gate_stride + first - shift, sizeof(T)),
                        *p_res = in(a.residual, at, sizeof(R));
    uint32_t unit_ask = id;
    auto ask_row = [&](int stage) {
        if (unit_ask < units) {
            const uint32_t to = (uint32_t)__cvta_generic_to_shared(rec0) + stage * kStage;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = e0 + c * span;
                const uint32_t t = (uint32_t)tid * V;
                const int64_t s = c * span;
                ask<T, V, SHIFTED>(to + kX, c, lane, p_x + s * sizeof(T), t * sizeof(T), e, n);
                if (GATE) ask<T, V, SHIFTED>(to + kZ, c, lane, p_gate + s * sizeof(T), t * sizeof(T), e, n);
                if (RES) ask<R, V, SHIFTED>(to + kR, c, lane, p_res + s * sizeof(R), t * sizeof(R), e, n);
            }
            unit_ask += a.slots;
            p_x += far * sizeof(T);
            if (GATE) p_gate += gate_far * sizeof(T);
            if (RES) p_res += far * sizeof(R);
        }
        copies_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) ask_row(s);
    // the weights' record; and zeros for vectors past the row's end, which nothing is copied into
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = e0 + c * span;
        float w[V] = {}, w2[V] = {};
        if (e < n) {
            row_weights<V, SHIFTED>(a.weight + first, e, n, w);
            if (RES && a.next_weight) row_weights<V, SHIFTED>(a.next_weight, e, n, w2);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            reinterpret_cast<float*>(wrec + piece<float, V>(c, k / 4, lane))[k % 4] = w[k];
            if (RES) reinterpret_cast<float*>(wrec + 32 * Rec::weight + piece<float, V>(c, k / 4, lane))[k % 4] = w2[k];
        }
        if (e >= n) {
            for (int s = 0; s < a.stages; ++s) {
                unsigned char* r = rec0 + s * kStage;
                clear_head<T, V>(r + kX, c, lane, V);
                if (GATE) clear_head<T, V>(r + kZ, c, lane, V);
                if (RES) clear_head<R, V>(r + kR, c, lane, V);
            }
        }
    }
    int stage = 0, turn = 0;   // sums alternate between two arrays
    for (uint32_t unit = id; unit < units; unit += a.slots, at += far) {
        unsigned char* const rec = rec0 + stage * kStage;
        if constexpr (kPairs) __syncwarp(mask);   // the row before is read
        ask_row(stage > 0 ? stage - 1 : a.stages - 1);   // where it lay
        if (++stage == a.stages) stage = 0;
        copies_wait(a.stages - 1);
        if constexpr (kPairs) __syncwarp(mask);
        if (SHIFTED && e0 < 0) {
            clear_head<T, V>(rec + kX, 0, lane, shift);
            if (GATE) clear_head<T, V>(rec + kZ, 0, lane, shift);
            if (RES) clear_head<R, V>(rec + kR, 0, lane, shift);
        }
        const uint32_t t = (uint32_t)tid * V;
        Two u[C][P], sum = both(0.f);
        RowMaxima m = {0, 0};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const Raw<T, V> xq = piece_vector<T, V>(rec + kX, c, lane);
            to_pairs(xq, u[c]);
            if (a.x_codes) m.a = max(m.a, magnitude(xq));
            if (GATE) {
                const Raw<T, V> zq = piece_vector<T, V>(rec + kZ, c, lane);
                if (a.x_codes) m.b = max(m.b, magnitude(zq));
                Two z[P];
                to_pairs(zq, z);
#pragma unroll
                for (int k = 0; k < P; ++k) u[c][k] = u[c][k] * (z[k] * sigmoid<T>(z[k]));
            }
#pragma unroll
            for (int k = 0; k < P; ++k) sum = fma(u[c][k], u[c][k], sum);
        }
        float ss[1] = {low(sum) + high(sum)};
        if (a.x_codes) {
            row_sum_maxima<LANES>(ss, m, part[turn]);
            const bool bad_x = m.a >= kInfBits, bad_z = m.b >= kInfBits;   // the same in all of the row's threads
            if (bad_x || bad_z) {
                m.a = m.b = 0;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    m.a = max(m.a, finite_magnitude(piece_vector<T, V>(rec + kX, c, lane)));
                    if (GATE) m.b = max(m.b, finite_magnitude(piece_vector<T, V>(rec + kZ, c, lane)));
                }
                m.a = row_maximum<LANES>(m.a, tops[0]);
                if (GATE) m.b = row_maximum<LANES>(m.b, tops[1]);
            }
            const uint32_t sx = pack_scale_bits(m.a), sz = pack_scale_bits(m.b);
            if (tid == 0) {
                a.x_scales[unit] = __uint_as_float(sx);
                if (GATE) a.gate_scales[unit] = __uint_as_float(sz);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                Two v[P];
                to_pairs(piece_vector<T, V>(rec + kX, c, lane), v);
                put_codes<V, SHIFTED>(static_cast<e4m3_t*>(a.x_codes) + at + c * span, t, e0 + c * span, n, v, pack_inverse(sx), bad_x);
                if (GATE) {
                    to_pairs(piece_vector<T, V>(rec + kZ, c, lane), v);
                    put_codes<V, SHIFTED>(static_cast<e4m3_t*>(a.gate_codes) + at + c * span, t, e0 + c * span, n, v, pack_inverse(sz), bad_z);
                }
            }
        } else {
            row_sum<LANES>(ss, part[turn]);
        }
        turn ^= 1;
        const Two rstd = both(rsqrt_of(ss[0] * a.inv_size + a.eps));
        unsigned char* const out = static_cast<unsigned char*>(a.out) + at * (int)sizeof(T);
        if constexpr (!RES) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                Two w[P];
                to_pairs(piece_vector<float, V>(wrec, c, lane), w);
#pragma unroll
                for (int k = 0; k < P; ++k) w[k] = u[c][k] * rstd * w[k];
                put<T, V, SHIFTED>(out + c * span * (int)sizeof(T), t * sizeof(T), e0 + c * span, n, mask, w);
            }
        } else {
            sum = both(0.f);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                Two w[P], r[P];
                to_pairs(piece_vector<float, V>(wrec, c, lane), w);
                to_pairs(piece_vector<R, V>(rec + kR, c, lane), r);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    u[c][k] = fma(both(a.scale), u[c][k] * rstd * w[k], r[k]);
                    sum = fma(u[c][k], u[c][k], sum);
                }
                put<R, V, SHIFTED>(static_cast<unsigned char*>(a.residual_out) + (at + c * span) * (int)sizeof(R), t * sizeof(R), e0 + c * span, n, mask,
                                   u[c]);
            }
            if (!a.next_weight) continue;
            ss[0] = low(sum) + high(sum);
            row_sum<LANES>(ss, part[turn]);
            turn ^= 1;
            const Two rstd2 = both(rsqrt_of(ss[0] * a.inv_size + a.eps));
            const bool codes = a.out_dtype == SSD_E4M3;
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                Two w[P];
                to_pairs(piece_vector<float, V>(wrec + 32 * Rec::weight, c, lane), w);
#pragma unroll
                for (int k = 0; k < P; ++k) u[c][k] = u[c][k] * rstd2 * w[k];
                if (codes) {
#pragma unroll
                    for (int k = 0; k < P; ++k)
                        for (const float f : {low(u[c][k]), high(u[c][k])}) {
                            const uint32_t b = __float_as_uint(f) & 0x7fffffffu;
                            if (b < kInfBits) top = max(top, b);
                        }
                } else {
                    put<T, V, SHIFTED>(out + c * span * (int)sizeof(T), t * sizeof(T), e0 + c * span, n, mask, u[c]);
                }
            }
            if (codes) {
                const uint32_t so = pack_scale_bits(row_maximum<LANES>(top, tops[0]));
                if (tid == 0) a.out_scales[unit] = __uint_as_float(so);
#pragma unroll
                for (int c = 0; c < C; ++c)
                    put_codes<V, SHIFTED>(static_cast<e4m3_t*>(a.out) + at + c * span, t, e0 + c * span, n, u[c], pack_inverse(so), true);
            }
        }
    }
}

// Where no vectors fit: single elements, a row a slot, all of it asked for before the first is used.
template <typename T, typename R, int E, int LANES, bool GATE, bool RES>
__global__ void __launch_bounds__(E == kNarrowElems ? 640 : 512) ssd_block_norm_loose(const __grid_constant__ BlockNormArgs a) {
    constexpr int V = 2, C = E / V, P = 1;   // pairs of single elements
    __shared__ RowPart part[2];
    __shared__ uint32_t tops[2][32];
    const int tid = LANES ? threadIdx.x % (LANES ? LANES : 32) : threadIdx.x, nt = LANES ? LANES : blockDim.x;
    const uint32_t unit = LANES ? blockIdx.x * a.units_per_cta + threadIdx.x / (LANES ? LANES : 32) : blockIdx.x;
    pdl_wait();
    if (unit >= a.units) return;   // all of a row's lanes
    const int n = a.size;
    const uint32_t row = a.groups == 1 ? unit : unit / (uint32_t)a.groups;
    const int64_t base = (int64_t)unit * n;
    const int first = (int)(unit - row * a.groups) * n;   // the group's first column
    const Place<V, false> place = {tid, nt, 0, n, n};
    Part<T, V, E, false> xq, zq;
    Part<R, V, E, false> rq;
    xq.load(static_cast<const T*>(a.x) + base, place);
    if (GATE) zq.load(static_cast<const T*>(a.gate) + row * a.gate_stride + first, place);
    if (RES) rq.load(static_cast<const R*>(a.residual) + base, place);
    Two u[C][P], sum = both(0.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        xq.get(c, u[c]);
        if (GATE) {
            Two z[P];
            zq.get(c, z);
            u[c][0] = u[c][0] * (z[0] * sigmoid<T>(z[0]));
        }
        sum = fma(u[c][0], u[c][0], sum);
    }
    float ss[1] = {low(sum) + high(sum)};
    if (a.x_codes) {
        RowMaxima m = {xq.top(), GATE ? zq.top() : 0};
        row_sum_maxima<LANES>(ss, m, part[0]);
        const bool bad_x = m.a >= kInfBits, bad_z = m.b >= kInfBits;   // the same in all of the row's threads
        if (bad_x || bad_z) {
            m.a = row_maximum<LANES>(xq.finite_top(), tops[0]);
            if (GATE) m.b = row_maximum<LANES>(zq.finite_top(), tops[1]);
        }
        const uint32_t sx = pack_scale_bits(m.a), sz = pack_scale_bits(m.b);
        if (tid == 0) {
            a.x_scales[unit] = __uint_as_float(sx);
            if (GATE) a.gate_scales[unit] = __uint_as_float(sz);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Two v[P];
            xq.get(c, v);
            store_codes<V, E, false>(static_cast<e4m3_t*>(a.x_codes) + base, place, c, v, pack_inverse(sx), bad_x);
            if (GATE) {
                zq.get(c, v);
                store_codes<V, E, false>(static_cast<e4m3_t*>(a.gate_codes) + base, place, c, v, pack_inverse(sz), bad_z);
            }
        }
    } else {
        row_sum<LANES>(ss, part[0]);
    }
    const Two rstd = both(rsqrt_of(ss[0] * a.inv_size + a.eps));
    if constexpr (!RES) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const Two w[P] = {u[c][0] * rstd * pair_weights(a.weight + first, place, c)};
            Part<T, V, E, false> q;
            q.set(c, w);
            q.store(static_cast<T*>(a.out) + base, place, c);
        }
    } else {
        sum = both(0.f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Two r[P];
            rq.get(c, r);
            u[c][0] = fma(both(a.scale), u[c][0] * rstd * pair_weights(a.weight, place, c), r[0]);
            sum = fma(u[c][0], u[c][0], sum);
            Part<R, V, E, false> q;
            q.set(c, u[c]);
            q.store(static_cast<R*>(a.residual_out) + base, place, c);
        }
        if (!a.next_weight) return;
        ss[0] = low(sum) + high(sum);
        row_sum<LANES>(ss, part[1]);
        const Two rstd2 = both(rsqrt_of(ss[0] * a.inv_size + a.eps));
        const bool codes = a.out_dtype == SSD_E4M3;
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            u[c][0] = u[c][0] * rstd2 * pair_weights(a.next_weight, place, c);
            if (codes) {
                for (const float f : {low(u[c][0]), high(u[c][0])}) {
                    const uint32_t b = __float_as_uint(f) & 0x7fffffffu;
                    if (b < kInfBits) top = max(top, b);
                }
            } else {
                Part<T, V, E, false> q;
                q.set(c, u[c]);
                q.store(static_cast<T*>(a.out) + base, place, c);
            }
        }
        if (!codes) return;
        const uint32_t so = pack_scale_bits(row_maximum<LANES>(top, tops[0]));
        if (tid == 0) a.out_scales[unit] = __uint_as_float(so);
#pragma unroll
        for (int c = 0; c < C; ++c)
            store_codes<V, E, false>(static_cast<e4m3_t*>(a.out) + base, place, c, u[c], pack_inverse(so), true);
    }
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Rows that a slot takes one after another, where there are enough for all SMs (block norm with its checkpoint 16384 x 2560 107 us, with
// 4 108, with 16 121; fp32 2048 columns 126, with 4 131; gate and norm 16384 x 5120 104, 103.5, 109).
constexpr int kSlotRows = 8;

template <typename T, typename R, int E, int LANES, bool SHIFTED, bool GATE, bool RES>
cudaError_t launch_ring(const BlockNormArgs& args, int threads, cudaStream_t st) {
    typedef Record<T, R, E, GATE, RES> Rec;
    BlockNormArgs a = args;
    auto kern = ssd_block_norm_kernel<T, R, E, LANES, SHIFTED, GATE, RES>;
    static std::atomic<uint8_t> ready[kMaxDevices];
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
    a.units_per_cta = LANES ? threads / (LANES ? LANES : 32) : 1;
    const int per_sm = fwd_threads_sm(E) / threads > 0 ? fwd_threads_sm(E) / threads : 1;
    // a multiple of 8 rows at a time
    const int64_t rows = a.units / a.groups, room = (int64_t)kAddNormSMs * per_sm * a.units_per_cta;
    int64_t each = a.units / room;
    each = each < 1 ? 1 : each > kSlotRows ? kSlotRows : each;
    int64_t lines = ((rows + each - 1) / each + 7) / 8 * 8;
    if (lines > rows) lines = rows;
    a.slots = (uint32_t)(lines * a.groups);
    const int stage = threads * Rec::bytes, weights = threads * Rec::weights;
    a.stages = lines < rows && weights + 2 * stage <= kSmemCta - kSmemOwn ? 2 : 1;
    if (weights + a.stages * stage > kSmemCta - kSmemOwn) return cudaErrorNotSupported;
    return launch_kernel(kern, (a.slots + a.units_per_cta - 1) / a.units_per_cta, (unsigned)threads, (size_t)weights + (size_t)a.stages * stage, st, true, a);
}

// Rows of up to 256 columns take lanes of a warp, others a CTA; 8 elements a thread up to 1024 columns, then 16.  65536 rows of bf16, 8 and
// 16 elements a thread: gate and norm with its checkpoint at 768 columns 65.5 and 66.6 us, at 1024 83.9 and 82.3, at 1280 111 and
// 102; with a residual and no gate 91.6 and 94.2, 119 and 121; fp32 1024 columns 139 and 143.
template <typename T, typename R, bool SHIFTED, bool GATE, bool RES>
cudaError_t launch_vectors(const BlockNormArgs& a, cudaStream_t st) {
    const int span = SHIFTED ? vector_span(a.size) : a.size;
    if (span <= 64) return launch_ring<T, R, kNarrowElems, 8, SHIFTED, GATE, RES>(a, 128, st);
    if (span <= 128) return launch_ring<T, R, kNarrowElems, 16, SHIFTED, GATE, RES>(a, 128, st);
    if (span <= 256) return launch_ring<T, R, kNarrowElems, 32, SHIFTED, GATE, RES>(a, 128, st);
    if (span <= 128 * kNarrowElems) return launch_ring<T, R, kNarrowElems, 0, SHIFTED, GATE, RES>(a, ((span + 7) / 8 + 31) / 32 * 32, st);
    return launch_ring<T, R, kWideElems, 0, SHIFTED, GATE, RES>(a, ((span + 15) / 16 + 31) / 32 * 32, st);
}

template <typename T, typename R, bool GATE, bool RES>
cudaError_t launch_loose(const BlockNormArgs& args, cudaStream_t st) {
    BlockNormArgs a = args;
    auto go = [&](auto kern, int lanes, int threads) {
        a.units_per_cta = lanes ? threads / lanes : 1;
        const unsigned grid = (unsigned)((a.units + a.units_per_cta - 1) / a.units_per_cta);
        return launch_kernel(kern, grid, (unsigned)threads, 0, st, true, a);
    };
    if (a.size <= 64) return go(ssd_block_norm_loose<T, R, kNarrowElems, 8, GATE, RES>, 8, 128);
    if (a.size <= 256) return go(ssd_block_norm_loose<T, R, kNarrowElems, 32, GATE, RES>, 32, 128);
    if (a.size <= 512 * kNarrowElems) return go(ssd_block_norm_loose<T, R, kNarrowElems, 0, GATE, RES>, 0, (a.size + 255) / 256 * 32);
    return go(ssd_block_norm_loose<T, R, kWideElems, 0, GATE, RES>, 0, (a.size + 511) / 512 * 32);
}

// Vectors where every array starts on 16 bytes (codes on a vector's), rows hold one at least and an SM's shared memory holds their
// records, single elements otherwise.
template <typename T, typename R, bool GATE, bool RES>
cudaError_t launch_typed(const BlockNormArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool shifted = a.size % V != 0, e4m3 = a.out_dtype == SSD_E4M3;
    const bool vectors = a.size >= V && vector_span(a.size) <= 512 * kWideElems && on16(a.x) && on16(a.residual) && on16(a.residual_out) &&
                         (e4m3 ? ((uintptr_t)a.out % V) == 0 : on16(a.out)) && ((uintptr_t)a.x_codes % V) == 0 &&
                         ((uintptr_t)a.gate_codes % V) == 0 && (shifted || (on16(a.weight) && on16(a.next_weight))) &&
                         (!GATE || (on16(a.gate) && (shifted ? a.gate_stride == (int64_t)a.size * a.groups : a.gate_stride % V == 0)));
    cudaError_t e = cudaErrorNotSupported;
    if (vectors) e = shifted ? launch_vectors<T, R, true, GATE, RES>(a, st) : launch_vectors<T, R, false, GATE, RES>(a, st);
    return e == cudaErrorNotSupported ? launch_loose<T, R, GATE, RES>(a, st) : e;
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& args, cudaStream_t st) {
    BlockNormArgs a = args;
    a.inv_size = 1.f / (float)a.size;
    if (!a.residual) return a.dtype == SSD_BF16 ? launch_typed<bf16_t, bf16_t, true, false>(a, st) : launch_typed<float, float, true, false>(a, st);
    if (a.dtype == SSD_F32) return a.gate ? launch_typed<float, float, true, true>(a, st) : launch_typed<float, float, false, true>(a, st);
    if (a.residual_dtype == SSD_F32)
        return a.gate ? launch_typed<bf16_t, float, true, true>(a, st) : launch_typed<bf16_t, float, false, true>(a, st);
    return a.gate ? launch_typed<bf16_t, bf16_t, true, true>(a, st) : launch_typed<bf16_t, bf16_t, false, true>(a, st);
}

}  // namespace ssd
