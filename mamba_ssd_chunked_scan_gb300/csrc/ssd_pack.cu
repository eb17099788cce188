// 8-bit rows (activation checkpoints):
//   ssd_pack_kernel     rows, or groups of each row's columns, as e4m3 numbers with a power of two each
//   ssd_unpack_kernel   what they stand for, in bf16 or fp32
//
// Both are bound by HBM: a unit (a row's group) stays in registers from its one read to its one write, since its
// scale needs all of it; unpacking is element by element over the flat array.
#include "ssd_kernels.h"
#include "ssd_rows.cuh"

namespace ssd {
namespace {

constexpr int kElems = 16;   // elements of a unit per thread

template <typename T, int V>
__global__ void __launch_bounds__(1024) ssd_pack_kernel(PackArgs a) {
    constexpr int C = kElems / V;
    __shared__ uint32_t part[2][32];
    const bool one_warp = a.units_per_cta > 1 || blockDim.x == 32;
    const int slot = one_warp ? threadIdx.x >> 5 : 0;
    const int tid = one_warp ? threadIdx.x & 31 : threadIdx.x;
    const int nt = one_warp ? 32 : blockDim.x;
    const int64_t unit = (int64_t)blockIdx.x * a.units_per_cta + slot;
    pdl_wait();
    if (unit >= a.units) return;   // whole warps of a many-unit CTA, which has no barrier
    const int64_t row = unit / a.groups;
    const int n = a.size;
    const T* x = static_cast<const T*>(a.x) + row * a.stride + (unit - row * a.groups) * n;
    e4m3_t* out = static_cast<e4m3_t*>(a.codes) + unit * n;
    Raw<T, V> r[C];
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (tid + c * nt) * V;
        r[c].zero();
        if (e < n) r[c].load(x + e);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) m = max(m, magnitude(r[c]));
    m = row_maximum(m, one_warp, part[0]);
    const bool bad = m >= kInfBits;   // the same in all of the unit's threads
    if (bad) {
        m = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) m = max(m, finite_magnitude(r[c]));
        m = row_maximum(m, one_warp, part[1]);
    }
    const uint32_t scale = pack_scale_bits(m);
    const float inv = pack_inverse(scale);
    if (tid == 0) a.scales[unit] = __uint_as_float(scale);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (tid + c * nt) * V;
        if (e < n) {
            float v[V];
            r[c].get(v);
            to_codes(v, inv, bad);
            Raw<e4m3_t, V> q;
            q.set(v);
            q.store(out + e);
        }
    }
}

// One thread per V elements of the output, whose rows lie together; codes' rows are `stride` apart.
template <typename T, int V>
__global__ void __launch_bounds__(256) ssd_unpack_kernel(PackArgs a) {
    pdl_trigger();
    pdl_wait();
    const int64_t per_row = ((int64_t)a.size * a.groups + V - 1) / V;
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = k / per_row;
    if (row >= a.units / a.groups) return;
    const int width = a.size * a.groups;
    const int e = (int)(k - row * per_row) * V;
    Raw<e4m3_t, V> q;
    q.load(static_cast<const e4m3_t*>(a.codes) + row * a.stride + e);
    float v[V];
    from_codes(q, v);
    const float* s = a.scales + row * a.groups;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= __ldg(s + (e + j) / a.size);
    Raw<T, V> o;
    o.set(v);
    o.store(static_cast<T*>(a.out) + row * width + e);
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T>
cudaError_t launch_pack_typed(PackArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.size % V == 0 && a.stride % V == 0 && on16(a.x) && ((uintptr_t)a.codes % V) == 0;
    int threads;
    if (a.size <= 32 * kElems) {
        a.units_per_cta = a.units < 4 ? (int)a.units : 4;
        threads = 32 * a.units_per_cta;
    } else {
        a.units_per_cta = 1;
        threads = ((a.size + kElems - 1) / kElems + 31) / 32 * 32;
    }
    const unsigned grid = (unsigned)((a.units + a.units_per_cta - 1) / a.units_per_cta);
    return launch_kernel(vec ? ssd_pack_kernel<T, V> : ssd_pack_kernel<T, 1>, grid, (unsigned)threads, 0, st, true, a);
}

template <typename T>
cudaError_t launch_unpack_typed(const PackArgs& a, cudaStream_t st) {
    const int64_t width = (int64_t)a.size * a.groups, rows = a.units / a.groups;
    const bool vec = width % 8 == 0 && a.stride % 8 == 0 && on16(a.out) && ((uintptr_t)a.codes % 8) == 0;
    const int64_t threads = rows * (vec ? width / 8 : width);
    return launch_kernel(vec ? ssd_unpack_kernel<T, 8> : ssd_unpack_kernel<T, 1>, (unsigned)((threads + 255) / 256), 256, 0, st, true, a);
}

}  // namespace

cudaError_t launch_pack(const PackArgs& args, cudaStream_t st) {
    PackArgs a = args;
    return a.dtype == SSD_BF16 ? launch_pack_typed<bf16_t>(a, st) : launch_pack_typed<float>(a, st);
}

cudaError_t launch_unpack(const PackArgs& a, cudaStream_t st) {
    return a.dtype == SSD_BF16 ? launch_unpack_typed<bf16_t>(a, st) : launch_unpack_typed<float>(a, st);
}

}  // namespace ssd
