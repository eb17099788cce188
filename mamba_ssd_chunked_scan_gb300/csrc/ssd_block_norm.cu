// The norm after a block, with the block's gate, the scaled residual addition and the next block's norm, in one pass:
//   ssd_block_norm_kernel   u = x silu(gate)  (or x)
//                           n = u rstd1 weight,                     rstd1 = 1 / sqrt(mean(u^2) + eps)
//                           h = residual + scale n                  (or, without a residual, out = n)
//                           out = h rstd2 next_weight,              rstd2 = 1 / sqrt(mean(h^2) + eps)
// and x and gate as 8-bit rows, for the backward pass.
//
// A row (a group of one, where the norm goes by groups: no residual then) is held in registers from its one read to its
// one write; h is normalised as it was summed, before its rounding to the residual's type.
#include "ssd_kernels.h"
#include "ssd_rows.cuh"

namespace ssd {
namespace {

constexpr int kElems = 16;   // elements of a row per thread

template <typename T, typename R, int V, bool GATE, bool RES>
__global__ void __launch_bounds__(512) ssd_block_norm_kernel(BlockNormArgs a) {
    constexpr int C = kElems / V;
    __shared__ RowPart part[2];
    __shared__ uint32_t tops[2][32];
    const bool one_warp = a.units_per_cta > 1 || blockDim.x == 32;
    const int slot = one_warp ? threadIdx.x >> 5 : 0;
    const int tid = one_warp ? threadIdx.x & 31 : threadIdx.x;
    const int nt = one_warp ? 32 : blockDim.x;
    const int64_t unit = (int64_t)blockIdx.x * a.units_per_cta + slot;
    pdl_wait();
    if (unit >= a.units) return;   // whole warps of a many-row CTA, which has no barrier
    const int n = a.size;
    const int64_t row = unit / a.groups;
    const int first = (int)(unit - row * a.groups) * n;   // the group's first column
    const size_t base = (size_t)unit * n;
    const T* x = static_cast<const T*>(a.x) + base;
    const T* gate = GATE ? static_cast<const T*>(a.gate) + row * a.gate_stride + first : nullptr;
    const R* res = RES ? static_cast<const R*>(a.residual) + base : nullptr;
    Raw<T, V> xr[C], gr[GATE ? C : 1];
    Raw<R, V> rr[RES ? C : 1];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (tid + c * nt) * V;
        xr[c].zero();
        if (GATE) gr[c].zero();
        if (RES) rr[c].zero();
        if (e < n) {
            xr[c].load(x + e);
            if (GATE) gr[c].load(gate + e);
            if (RES) rr[c].load(res + e);
        }
    }
    float u[C][V];
    float ss[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
        xr[c].get(u[c]);
        if (GATE) {
            float g[V];
            gr[c].get(g);
#pragma unroll
            for (int k = 0; k < V; ++k) u[c][k] *= g[k] * sigmoid<T>(g[k]);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) ss[0] = fmaf(u[c][k], u[c][k], ss[0]);
    }
    if (a.x_codes) {
        RowMaxima m = {0, 0};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            m.a = max(m.a, magnitude(xr[c]));
            if (GATE) m.b = max(m.b, magnitude(gr[c]));
        }
        row_sum_maxima(ss, m, one_warp, part[0]);
        const bool bad_x = m.a >= kInfBits, bad_g = m.b >= kInfBits;   // the same in all of the row's threads
        if (bad_x || bad_g) {
            m.a = m.b = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                m.a = max(m.a, finite_magnitude(xr[c]));
                if (GATE) m.b = max(m.b, finite_magnitude(gr[c]));
            }
            m.a = row_maximum(m.a, one_warp, tops[0]);
            m.b = row_maximum(m.b, one_warp, tops[1]);
        }
        const uint32_t sx = pack_scale_bits(m.a), sg = pack_scale_bits(m.b);
        if (tid == 0) {
            a.x_scales[unit] = __uint_as_float(sx);
            if (GATE) a.gate_scales[unit] = __uint_as_float(sg);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (tid + c * nt) * V;
            if (e < n) {
                float v[V];
                Raw<e4m3_t, V> q;
                xr[c].get(v);
                to_codes(v, pack_inverse(sx), bad_x);
                q.set(v);
                q.store(static_cast<e4m3_t*>(a.x_codes) + base + e);
                if (GATE) {
                    gr[c].get(v);
                    to_codes(v, pack_inverse(sg), bad_g);
                    q.set(v);
                    q.store(static_cast<e4m3_t*>(a.gate_codes) + base + e);
                }
            }
        }
    } else {
        row_sums(ss, one_warp, part[0]);
    }
    const float rstd = rsqrt_of(ss[0] * a.inv_size + a.eps);
    float hh = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (tid + c * nt) * V;
        if (e < n) {
            float w[V];
            row_weights<V, false>(a.weight + first, e, n, w);
            if (RES) {
                float r[V];
                rr[c].get(r);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    u[c][k] = fmaf(a.scale, u[c][k] * rstd * w[k], r[k]);
                    hh = fmaf(u[c][k], u[c][k], hh);
                }
                Raw<R, V> q;
                q.set(u[c]);
                q.store(static_cast<R*>(a.residual_out) + base + e);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) u[c][k] = u[c][k] * rstd * w[k];
                Raw<T, V> q;
                q.set(u[c]);
                q.store(static_cast<T*>(a.out) + base + e);
            }
        }
    }
    if constexpr (RES) {
        if (!a.next_weight) return;
        float s[1] = {hh};
        row_sums(s, one_warp, part[1]);
        const float rstd2 = rsqrt_of(s[0] * a.inv_size + a.eps);
        const bool codes = a.out_dtype == SSD_E4M3;
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (tid + c * nt) * V;
            if (e < n) {
                float w[V];
                row_weights<V, false>(a.next_weight, e, n, w);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    u[c][k] = u[c][k] * rstd2 * w[k];
                    const uint32_t b = __float_as_uint(u[c][k]) & 0x7fffffffu;
                    if (b < kInfBits) top = max(top, b);
                }
                if (!codes) {
                    Raw<T, V> q;
                    q.set(u[c]);
                    q.store(static_cast<T*>(a.out) + base + e);
                }
            }
        }
        if (!codes) return;
        const uint32_t so = pack_scale_bits(row_maximum(top, one_warp, tops[0]));
        if (tid == 0) a.out_scales[unit] = __uint_as_float(so);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (tid + c * nt) * V;
            if (e < n) {
                Raw<e4m3_t, V> q;
                to_codes(u[c], pack_inverse(so), true);
                q.set(u[c]);
                q.store(static_cast<e4m3_t*>(a.out) + base + e);
            }
        }
    }
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, typename R, bool RES>
cudaError_t launch_typed(const BlockNormArgs& a, unsigned grid, unsigned threads, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.size % V == 0 && on16(a.x) && on16(a.residual) && on16(a.residual_out) && on16(a.weight) && on16(a.next_weight) &&
                     on16(a.out) && ((uintptr_t)a.x_codes % V) == 0 && ((uintptr_t)a.gate_codes % V) == 0 &&
                     (!a.gate || (a.gate_stride % V == 0 && on16(a.gate)));
    if (a.gate)
        return launch_kernel(vec ? ssd_block_norm_kernel<T, R, V, true, RES> : ssd_block_norm_kernel<T, R, 1, true, RES>, grid, threads, 0,
                             st, true, a);
    if constexpr (RES)
        return launch_kernel(vec ? ssd_block_norm_kernel<T, R, V, false, RES> : ssd_block_norm_kernel<T, R, 1, false, RES>, grid, threads, 0,
                             st, true, a);
    return cudaErrorInvalidValue;   // a norm without gate or residual is ssd_add_norm's
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& args, cudaStream_t st) {
    BlockNormArgs a = args;
    a.inv_size = 1.f / (float)a.size;
    unsigned threads;
    if (a.size <= 32 * kElems) {
        a.units_per_cta = a.units < 4 ? (int)a.units : 4;
        threads = 32 * a.units_per_cta;
    } else {
        a.units_per_cta = 1;
        threads = ((a.size + kElems - 1) / kElems + 31) / 32 * 32;
    }
    const unsigned grid = (unsigned)((a.units + a.units_per_cta - 1) / a.units_per_cta);
    if (!a.residual)
        return a.dtype == SSD_BF16 ? launch_typed<bf16_t, bf16_t, false>(a, grid, threads, st) : launch_typed<float, float, false>(a, grid, threads, st);
    if (a.dtype == SSD_BF16)
        return a.residual_dtype == SSD_F32 ? launch_typed<bf16_t, float, true>(a, grid, threads, st)
                                           : launch_typed<bf16_t, bf16_t, true>(a, grid, threads, st);
    return launch_typed<float, float, true>(a, grid, threads, st);
}

}  // namespace ssd
