// 8-bit rows (activation checkpoints):
//   ssd_pack_kernel     rows, or groups of each row's columns, as e4m3 numbers with a power of two each
//   ssd_unpack_kernel   what they stand for, in bf16 or fp32
//
// Both are bound by HBM: a unit (a row's group) stays in registers from its one read to its one write, since its
// scale needs all of it (16384 x 5120 bf16 columns of a wider matrix 40 us, 93 % of the copy's rate; 4096 columns of fp32 49 us, all
// of it); unpacking goes by 16 elements of the flat array, whatever the rows' width (16384 x 2560 to bf16 20 us, 91 %; to fp32 45 us,
// 69 %, and 4099 x 2557 12 us, 63 %: a thread's four 16-byte stores lie 64 bytes from its neighbour's, so that each store instruction
// writes half of every sector it touches).
#include "ssd_kernels.h"
#include "ssd_unpack.cuh"

namespace ssd {
namespace {

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, int V, int E, int LANES, bool SHIFTED>
__global__ void __launch_bounds__(1024) ssd_pack_kernel(const __grid_constant__ PackArgs a) {
    __shared__ uint32_t part[2][32];
    const int tid = LANES ? threadIdx.x % (LANES ? LANES : 32) : threadIdx.x, nt = LANES ? LANES : blockDim.x;
    const uint32_t unit = LANES ? blockIdx.x * a.units_per_cta + threadIdx.x / (LANES ? LANES : 32) : blockIdx.x;
    pdl_wait();
    if (unit >= a.units) return;   // all of a unit's lanes
    const int n = a.size;
    const uint32_t row = a.groups == 1 ? unit : unit / (uint32_t)a.groups;
    const int64_t base = (int64_t)unit * n;
    const Place<V, SHIFTED> place = {tid, nt, SHIFTED ? (int)(base & (V - 1)) : 0, n, (a.units - unit) * n};
    Part<T, V, E, SHIFTED> q;
    q.load(static_cast<const T*>(a.x) + row * a.stride + (int64_t)(unit - row * a.groups) * n, place);
    uint32_t m = row_maximum<LANES>(q.top(), part[0]);
    const bool bad = m >= kInfBits;   // the same in all of the unit's threads
    if (bad) m = row_maximum<LANES>(q.finite_top(), part[1]);
    const uint32_t scale = pack_scale_bits(m);
    if (tid == 0) a.scales[unit] = __uint_as_float(scale);
#pragma unroll
    for (int c = 0; c < E / V; ++c) {
        Two v[V / 2];
        q.get(c, v);
        store_codes<V, E, SHIFTED>(static_cast<e4m3_t*>(a.codes) + base, place, c, v, pack_inverse(scale), bad);
    }
}

template <typename T>
__global__ void __launch_bounds__(kFlatThreads) ssd_unpack_kernel(const __grid_constant__ PackArgs a) {
    pdl_trigger();
    pdl_wait();
    unpack_flat<T>(a, blockIdx.x);
}

// Any alignment, and codes whose rows are `stride` apart: V elements of an output row per thread.
template <typename T, int V>
__global__ void __launch_bounds__(256) ssd_unpack_rows_kernel(const __grid_constant__ PackArgs a) {
    pdl_trigger();
    pdl_wait();
    const int width = a.size * a.groups, per_row = (width + 256 * V - 1) / (256 * V);   // CTAs of a row
    const int64_t row = blockIdx.x / per_row;
    const int e = ((int)(blockIdx.x - row * per_row) * 256 + (int)threadIdx.x) * V;
    if (e >= width) return;
    Raw<e4m3_t, V> q;
    q.load(static_cast<const e4m3_t*>(a.codes) + row * a.stride + e);
    float v[V];
    from_codes(q, v);
    const float* s = a.scales + row * a.groups;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float f = __ldg(s + (a.groups == 1 ? 0 : (e + j) / a.size));
        v[j] *= a.power_only ? scale_power(f) : f;
    }
    Raw<T, V> o;
    o.set(v);
    o.store(static_cast<T*>(a.out) + row * width + e);
}


template <typename T, int V, bool SHIFTED>
cudaError_t launch_pack_shape(PackArgs& a, cudaStream_t st) {
    const int span = SHIFTED ? a.size + V - 1 : a.size;   // columns that the vectors of a unit may span
    auto go = [&](auto kern, int lanes, int threads) {
        a.units_per_cta = lanes ? threads / lanes : 1;
        const unsigned grid = (unsigned)((a.units + a.units_per_cta - 1) / a.units_per_cta);
        return launch_kernel(kern, grid, (unsigned)threads, 0, st, true, a);
    };
    // Lanes of a warp for up to 256 columns (131072 x 256 bf16 18 us, a CTA of a warp each 67); then CTAs, of 16 elements a thread: with 8
    // 16384 x 5120 56 us instead of 40, 65536 x 1024 35.3 instead of 34.7.
    if (span <= 64) return go(ssd_pack_kernel<T, V, 8, 8, SHIFTED>, 8, 128);
    if (span <= 128) return go(ssd_pack_kernel<T, V, 8, 16, SHIFTED>, 16, 128);
    if (span <= 256) return go(ssd_pack_kernel<T, V, 8, 32, SHIFTED>, 32, 128);
    return go(ssd_pack_kernel<T, V, 16, 0, SHIFTED>, 0, ((span + 15) / 16 + 31) / 32 * 32);
}

// Vectors where both arrays start on 16 bytes (codes on a vector's) and units hold one at least, single elements otherwise.
template <typename T>
cudaError_t launch_pack_typed(PackArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool shifted = a.size % V != 0;
    const bool vectors = a.size >= V && (!shifted || a.size + V - 1 <= 1024 * 16) && on16(a.x) && ((uintptr_t)a.codes % V) == 0 &&
                         (shifted ? a.stride == (int64_t)a.size * a.groups : a.stride % V == 0);
    if (!vectors) return launch_pack_shape<T, 2, false>(a, st);
    return shifted ? launch_pack_shape<T, V, true>(a, st) : launch_pack_shape<T, V, false>(a, st);
}

template <typename T>
cudaError_t launch_unpack_typed(const PackArgs& a, cudaStream_t st) {
    const int64_t width = (int64_t)a.size * a.groups, rows = a.units / a.groups;
    if (const unsigned ctas = unpack_flat_ctas(a)) return launch_kernel(ssd_unpack_kernel<T>, ctas, kFlatThreads, 0, st, true, a);
    const bool vec = width % 8 == 0 && a.stride % 8 == 0 && on16(a.out) && ((uintptr_t)a.codes % 8) == 0;
    const int64_t ctas = rows * ((width + 256 * (vec ? 8 : 1) - 1) / (256 * (vec ? 8 : 1)));
    return launch_kernel(vec ? ssd_unpack_rows_kernel<T, 8> : ssd_unpack_rows_kernel<T, 1>, (unsigned)ctas, 256, 0, st, true, a);
}

}  // namespace

unsigned unpack_flat_ctas(const PackArgs& a) {
    if (a.stride != (int64_t)a.size * a.groups || !on16(a.codes) || !on16(a.out)) return 0;
    return (unsigned)((a.units * a.size + kFlatThreads * kFlat - 1) / (kFlatThreads * kFlat));
}

cudaError_t launch_pack(const PackArgs& args, cudaStream_t st) {
    PackArgs a = args;
    return a.dtype == SSD_BF16 ? launch_pack_typed<bf16_t>(a, st) : launch_pack_typed<float>(a, st);
}

cudaError_t launch_unpack(const PackArgs& a, cudaStream_t st) {
    return a.dtype == SSD_BF16 ? launch_unpack_typed<bf16_t>(a, st) : launch_unpack_typed<float>(a, st);
}

}  // namespace ssd
