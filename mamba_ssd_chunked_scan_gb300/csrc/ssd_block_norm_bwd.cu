// Gradients of the norm after a block (ssd_block_norm_kernel's formula) and of the gate and grouped norm after the scan:
//   ssd_block_norm_bwd_kernel   p2 = next_weight dout, hh = h rstd2:  dh = dres + rstd2 (p2 - hh mean(p2 hh))
//                               p1 = scale dh weight,  uh = u rstd1:  du = rstd1 (p1 - uh mean(p1 uh))
//                               dx = du silu(gate),  dgate = du x s (1 + gate (1 - s)),  s = 1 / (1 + e^-gate)
//                               and each row slot's shares of  dweight = sum scale dh uh,  dnext_weight = sum dout hh
//   (without a residual: scale dh is dout itself)
//
// u and both rstd are recomputed from x, gate and h, which may be 8-bit rows.  A grid as large as the GPU holds at
// once walks the rows, so that the shares stay few; ssd_share_sum adds them in a fixed order.
#include "ssd_kernels.h"
#include "ssd_rows.cuh"

namespace ssd {
namespace {

// Elements of a row that a thread reads from one operand: of type T, or 8-bit codes times the row's scale.
template <typename T, int V>
__device__ __forceinline__ void take(const void* p, size_t at, bool packed, float scale, float (&v)[V]) {
    if (packed) {
        Raw<e4m3_t, V> q;
        q.load(static_cast<const e4m3_t*>(p) + at);
        from_codes(q, v);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] *= scale;
    } else {
        Raw<T, V> q;
        q.load(static_cast<const T*>(p) + at);
        q.get(v);
    }
}

template <typename T, typename R, int V, int E, bool GATE, bool RES>
__global__ void __launch_bounds__(512) ssd_block_norm_bwd_kernel(BlockNormBwdArgs a) {
    constexpr int C = E / V;
    __shared__ float4 part[2][16];
    const bool one_warp = a.slots_per_cta > 1 || blockDim.x == 32;
    const int slot = one_warp ? threadIdx.x >> 5 : 0;
    const int tid = one_warp ? threadIdx.x & 31 : threadIdx.x;
    const int nt = one_warp ? 32 : blockDim.x;
    const int id = blockIdx.x * a.slots_per_cta + slot;
    pdl_trigger();
    pdl_wait();
    if (id >= a.slots) return;   // whole warps of a many-slot CTA, which has no barrier
    const int n = a.size;
    const int line = id / a.groups, first = (id - line * a.groups) * n;   // the slot's first row, and its group's first column
    const int64_t step = a.slots / a.groups;
    const bool next = RES && a.dout;
    float dw[C][V], dn[RES ? C : 1][V];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            dw[c][k] = 0.f;
            if (RES) dn[c][k] = 0.f;
        }
    int turn = 0;
    for (int64_t row = line; row < a.rows; row += step) {
        const int64_t unit = row * a.groups + first / n;
        const size_t base = (size_t)unit * n, gbase = GATE ? (size_t)row * a.gate_stride + first : 0;
        const float xs = a.x_scales ? __ldg(a.x_scales + unit) : 1.f;
        const float gs = GATE && a.gate_scales ? __ldg(a.gate_scales + unit) : 1.f;
        const float hs = RES && a.h_scales ? __ldg(a.h_scales + unit) : 1.f;
        // u (kept), and what the first means need
        float u[C][V], sg[GATE ? C : 1][V], g1[C][V];   // g1: the gradient of n = u rstd1 weight
        RowSums s = {0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (tid + c * nt) * V;
#pragma unroll
            for (int k = 0; k < V; ++k) u[c][k] = g1[c][k] = 0.f;
            if (e >= n) continue;
            take<T>(a.x, base + e, a.x_scales, xs, u[c]);
            if (GATE) {
                float g[V];
                take<T>(a.gate, gbase + e, a.gate_scales, gs, g);
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
                    take<R>(a.h, base + e, a.h_scales, hs, h);
                    take<T>(a.dout, base + e, false, 1.f, d);
                    row_weights<V, false>(a.next_weight, e, n, w);
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        s.b = fmaf(h[k], h[k], s.b);
                        s.c = fmaf(d[k] * w[k], h[k], s.c);
                    }
                }
            } else {
                take<T>(a.dout, base + e, false, 1.f, g1[c]);
                row_weights<V, false>(a.weight + first, e, n, w);
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
                const int e = (tid + c * nt) * V;
                if (e >= n) continue;
                float dh[V], w[V];
                take<R>(a.dres, base + e, false, 1.f, dh);
                if (next) {
                    float h[V], d[V];
                    take<R>(a.h, base + e, a.h_scales, hs, h);
                    take<T>(a.dout, base + e, false, 1.f, d);
                    row_weights<V, false>(a.next_weight, e, n, w);
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        dh[k] = fmaf(rstd2, fmaf(d[k], w[k], -h[k] * mean2), dh[k]);
                        dn[c][k] = fmaf(d[k], h[k] * rstd2, dn[c][k]);
                    }
                }
                Raw<R, V> q;
                q.set(dh);
                q.store(static_cast<R*>(a.dres_out) + base + e);
                row_weights<V, false>(a.weight, e, n, w);
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
            const int e = (tid + c * nt) * V;
            if (e >= n) continue;
            float w[V], du[V];
            row_weights<V, false>(a.weight + first, e, n, w);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                du[k] = rstd * fmaf(g1[c][k], w[k], -u[c][k] * mean1);
                dw[c][k] = fmaf(g1[c][k], u[c][k] * rstd, dw[c][k]);
            }
            if (!RES && a.out) {
                Raw<T, V> q;
                float o[V];
#pragma unroll
                for (int k = 0; k < V; ++k) o[k] = u[c][k] * rstd * w[k];
                q.set(o);
                q.store(static_cast<T*>(a.out) + base + e);
            }
            if (GATE) {
                float x[V], g[V], dg[V];
                take<T>(a.x, base + e, a.x_scales, xs, x);
                take<T>(a.gate, gbase + e, a.gate_scales, gs, g);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float b = g[k] * sg[c][k];
                    dg[k] = du[k] * x[k] * fmaf(sg[c][k], 1.f - b, b);   // s + gate s (1 - s)
                    du[k] *= b;
                }
                Raw<T, V> q;
                q.set(dg);
                q.store(static_cast<T*>(a.dgate) + (size_t)row * a.dgate_stride + first + e);
            }
            Raw<T, V> q;
            q.set(du);
            q.store(static_cast<T*>(a.dx) + base + e);
        }
    }
    const int width = n * a.groups, columns = RES && a.next_weight ? 2 * width : width;
    float* share = a.shares + (size_t)line * columns + first;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (tid + c * nt) * V;
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (e < n) {
                share[e + k] = dw[c][k];
                if (RES && a.next_weight) share[width + e + k] = dn[c][k];
            }
    }
}

struct Plan {
    int threads, slots_per_cta, slots, grid;
};

constexpr int kElems = 16;
constexpr int kThreadsSM = 512;

Plan plan(int64_t rows, int size, int groups) {
    Plan p;
    int cta_slots = 1;
    if (size <= 32 * kElems) {
        cta_slots = 4;
        p.threads = 128;
    } else {
        p.threads = ((size + kElems - 1) / kElems + 31) / 32 * 32;
    }
    const int per_sm = kThreadsSM / p.threads > 0 ? kThreadsSM / p.threads : 1;
    int64_t lines = (int64_t)kAddNormSMs * per_sm * cta_slots / groups / 8 * 8;
    if (lines < 8) lines = 8;
    if (lines > rows) lines = rows;
    p.slots = (int)lines * groups;
    p.slots_per_cta = p.slots < cta_slots ? p.slots : cta_slots;
    if (cta_slots > 1) p.threads = 32 * p.slots_per_cta;
    p.grid = (p.slots + p.slots_per_cta - 1) / p.slots_per_cta;
    return p;
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, typename R, bool GATE, bool RES>
cudaError_t launch_typed(const BlockNormBwdArgs& a, const Plan& p, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    auto aligned = [&](const void* q, bool packed) { return packed ? ((uintptr_t)q % V) == 0 : on16(q); };
    const bool vec = a.size % V == 0 && aligned(a.x, a.x_scales) && aligned(a.h, a.h_scales) && on16(a.dout) && on16(a.dres) && on16(a.dres_out) &&
                     on16(a.dx) && on16(a.out) && on16(a.weight) && on16(a.next_weight) &&
                     (!GATE || (aligned(a.gate, a.gate_scales) && on16(a.dgate) && a.gate_stride % V == 0 && a.dgate_stride % V == 0));
    return launch_kernel(vec ? ssd_block_norm_bwd_kernel<T, R, V, kElems, GATE, RES> : ssd_block_norm_bwd_kernel<T, R, 1, kElems, GATE, RES>,
                         (unsigned)p.grid, (unsigned)p.threads, 0, st, true, a);
}

}  // namespace

int64_t block_norm_bwd_lines(int64_t rows, int size, int groups) { return plan(rows, size, groups).slots / groups; }

cudaError_t launch_block_norm_bwd(const BlockNormBwdArgs& args, cudaStream_t st) {
    BlockNormBwdArgs a = args;
    const Plan p = plan(a.rows, a.size, a.groups);
    a.slots = p.slots;
    a.slots_per_cta = p.slots_per_cta;
    a.inv_size = 1.f / (float)a.size;
    cudaError_t e;
    if (!a.dres)
        e = a.dtype == SSD_BF16 ? launch_typed<bf16_t, bf16_t, true, false>(a, p, st) : launch_typed<float, float, true, false>(a, p, st);
    else if (a.dtype == SSD_F32)
        e = a.gate ? launch_typed<float, float, true, true>(a, p, st) : launch_typed<float, float, false, true>(a, p, st);
    else if (a.residual_dtype == SSD_F32)
        e = a.gate ? launch_typed<bf16_t, float, true, true>(a, p, st) : launch_typed<bf16_t, float, false, true>(a, p, st);
    else
        e = a.gate ? launch_typed<bf16_t, bf16_t, true, true>(a, p, st) : launch_typed<bf16_t, bf16_t, false, true>(a, p, st);
    if (e != cudaSuccess) return e;
    const int width = a.size * a.groups;
    return launch_share_sum(a.shares, p.slots / a.groups, width, a.next_weight ? 2 * width : width, a.dweight, a.dnext_weight, st);
}

}  // namespace ssd
