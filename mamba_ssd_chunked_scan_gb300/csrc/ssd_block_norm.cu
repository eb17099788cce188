// The norm after a block, with the block's gate, the scaled residual addition and the next block's norm, in one pass:
//   ssd_block_norm_kernel   u = x silu(gate)  (or x)
//                           n = u rstd1 weight,                     rstd1 = 1 / sqrt(mean(u^2) + eps)
//                           h = residual + scale n                  (or, without a residual, out = n)
//                           out = h rstd2 next_weight,              rstd2 = 1 / sqrt(mean(h^2) + eps)
// and x and gate as 8-bit rows, for the backward pass.
//
// A row (a group of one, where the norm goes by groups: no residual then) is held in registers from its one read to its
// one write; h is normalised as it was summed, before its rounding to the residual's type.  Groups of up to 256 columns
// share warps; what a row's threads take is in ssd_rows.cuh.
#include "ssd_kernels.h"
#include "ssd_rows.cuh"

namespace ssd {
namespace {

template <typename T, typename R, int V, int E, int LANES, bool SHIFTED, bool GATE, bool RES>
__global__ void __launch_bounds__(512) ssd_block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
    constexpr int C = E / V, P = V / 2;
    __shared__ RowPart part[2];
    __shared__ uint32_t tops[2][32];
    const int tid = LANES ? threadIdx.x % (LANES ? LANES : 32) : threadIdx.x, nt = LANES ? LANES : blockDim.x;
    const int64_t unit = LANES ? (int64_t)blockIdx.x * a.units_per_cta + threadIdx.x / (LANES ? LANES : 32) : blockIdx.x;
    pdl_wait();
    if (unit >= a.units) return;   // all of a row's lanes
    const int n = a.size;
    const int64_t row = unit / a.groups, base = unit * n;
    const int first = (int)(unit - row * a.groups) * n;   // the group's first column
    const Place<V, SHIFTED> place = {tid, nt, SHIFTED ? (int)(base % V) : 0, n, (a.units - unit) * n};
    Part<T, V, E, SHIFTED> xq, zq;
    Part<R, V, E, SHIFTED> rq;
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
#pragma unroll
            for (int k = 0; k < P; ++k) u[c][k] = u[c][k] * (z[k] * sigmoid<T>(z[k]));
        }
#pragma unroll
        for (int k = 0; k < P; ++k) sum = fma(u[c][k], u[c][k], sum);
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
            store_codes<V, E, SHIFTED>(static_cast<e4m3_t*>(a.x_codes) + base, place, c, v, pack_inverse(sx), bad_x);
            if (GATE) {
                zq.get(c, v);
                store_codes<V, E, SHIFTED>(static_cast<e4m3_t*>(a.gate_codes) + base, place, c, v, pack_inverse(sz), bad_z);
            }
        }
    } else {
        row_sum<LANES>(ss, part[0]);
    }
    const Two rstd = both(rsqrt_of(ss[0] * a.inv_size + a.eps));
    if constexpr (!RES) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Two w[P];
            weights_of<V, SHIFTED>(a.weight + first, place, c, w);
#pragma unroll
            for (int k = 0; k < P; ++k) w[k] = u[c][k] * rstd * w[k];
            Part<T, V, E, SHIFTED> q;
            q.set(c, w);
            q.store(static_cast<T*>(a.out) + base, place, c);
        }
    } else {
        sum = both(0.f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Two w[P], r[P];
            weights_of<V, SHIFTED>(a.weight, place, c, w);
            rq.get(c, r);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                u[c][k] = fma(both(a.scale), u[c][k] * rstd * w[k], r[k]);
                sum = fma(u[c][k], u[c][k], sum);
            }
            Part<R, V, E, SHIFTED> q;
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
            Two w[P];
            weights_of<V, SHIFTED>(a.next_weight, place, c, w);
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
                Part<T, V, E, SHIFTED> q;
                q.set(c, u[c]);
                q.store(static_cast<T*>(a.out) + base, place, c);
            }
        }
        if (!codes) return;
        const uint32_t so = pack_scale_bits(row_maximum<LANES>(top, tops[0]));
        if (tid == 0) a.out_scales[unit] = __uint_as_float(so);
#pragma unroll
        for (int c = 0; c < C; ++c)
            store_codes<V, E, SHIFTED>(static_cast<e4m3_t*>(a.out) + base, place, c, u[c], pack_inverse(so), true);
    }
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, typename R, int V, bool SHIFTED, bool GATE, bool RES>
cudaError_t launch_shape(const BlockNormArgs& args, cudaStream_t st) {
    BlockNormArgs a = args;
    const int span = SHIFTED ? a.size + V - 1 : a.size;   // columns that the vectors of a row may span
    auto go = [&](auto kern, int lanes, int threads) {
        a.units_per_cta = lanes ? threads / lanes : 1;
        const unsigned grid = (unsigned)((a.units + a.units_per_cta - 1) / a.units_per_cta);
        return launch_kernel(kern, grid, (unsigned)threads, 0, st, true, a);
    };
    if (span <= 64) return go(ssd_block_norm_kernel<T, R, V, 8, 8, SHIFTED, GATE, RES>, 8, 128);
    if (span <= 128) return go(ssd_block_norm_kernel<T, R, V, 8, 16, SHIFTED, GATE, RES>, 16, 128);
    if (span <= 256) return go(ssd_block_norm_kernel<T, R, V, 8, 32, SHIFTED, GATE, RES>, 32, 128);
    return go(ssd_block_norm_kernel<T, R, V, 16, 0, SHIFTED, GATE, RES>, 0, ((span + 15) / 16 + 31) / 32 * 32);
}

// Vectors where every array starts on 16 bytes (codes on a vector's) and rows hold one at least, single elements otherwise.
template <typename T, typename R, bool GATE, bool RES>
cudaError_t launch_typed(const BlockNormArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool shifted = a.size % V != 0, e4m3 = a.out_dtype == SSD_E4M3;
    const bool vectors = a.size >= V && (!shifted || a.size + V - 1 <= 512 * 16) && on16(a.x) && on16(a.residual) && on16(a.residual_out) &&
                         (e4m3 ? ((uintptr_t)a.out % V) == 0 : on16(a.out)) && ((uintptr_t)a.x_codes % V) == 0 &&
                         ((uintptr_t)a.gate_codes % V) == 0 && (shifted || (on16(a.weight) && on16(a.next_weight))) &&
                         (!GATE || (on16(a.gate) && (shifted ? a.gate_stride == (int64_t)a.size * a.groups : a.gate_stride % V == 0)));
    if (!vectors) return launch_shape<T, R, 2, false, GATE, RES>(a, st);
    return shifted ? launch_shape<T, R, V, true, GATE, RES>(a, st) : launch_shape<T, R, V, false, GATE, RES>(a, st);
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
