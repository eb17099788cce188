// Rows of activations in the norms around a block and their 8-bit checkpoints (sm_103a): how a row's
// threads reduce over it, and how it becomes e4m3 numbers with a scale.
//
// An 8-bit row is code * scale with scale = 2^s the smallest power of two for which max |x| <= 448 scale (at least
// 2^-108).  e4m3 is a floating type, so a power of two costs no precision against max / 448, and everything about it
// is exact but the one rounding of x / scale: the quotient, the value code * scale (four significant bits, a bf16
// number), and what the backward passes make of it.  An element that is infinite or NaN becomes NaN by itself; the
// scale is that of the others.
#pragma once
#include "ssd_common.cuh"
#include "ssd_vec.cuh"

namespace ssd {

constexpr uint32_t kInfBits = 0x7f800000u;    // magnitudes of fp32 numbers as integers: finite ones are below
constexpr int kPackMinExp = -108;             // of a scale: 2^-9 of it is still a normal number

// The scale's bits for a largest magnitude `amax` (the bits of a finite fp32 number): 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t pack_scale_bits(uint32_t amax) {
    const int e = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u);
    return (uint32_t)(e < 127 + kPackMinExp ? 127 + kPackMinExp : e) << 23;
}
// Its reciprocal, a normal number too (exponents of scales are -108 to 120).
__device__ __forceinline__ float pack_inverse(uint32_t scale_bits) { return __uint_as_float((254u << 23) - scale_bits); }

// Largest magnitude of V elements as fp32 bits, infinities and NaNs as they are (at least kInfBits).
template <typename T, int V>
__device__ __forceinline__ uint32_t magnitude(const Raw<T, V>& r) {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r.w);
#pragma unroll
        for (int k = 0; k < V; ++k) m = max(m, w[k] & 0x7fffffffu);
    } else if constexpr (V == 1) {
        m = (uint32_t)(r.w & 0x7fffu) << 16;
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r.w);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) m = __vmaxu2(m, w[k] & 0x7fff7fffu);
        m = max(m & 0xffff0000u, m << 16);
    }
    return m;
}
// The same over the finite ones alone.
template <typename T, int V>
__device__ __forceinline__ uint32_t finite_magnitude(const Raw<T, V>& r) {
    float v[V];
    r.get(v);
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const uint32_t b = __float_as_uint(v[k]) & 0x7fffffffu;
        if (b < kInfBits) m = max(m, b);
    }
    return m;
}

// V elements as codes; `bad`: some element of the row is infinite or NaN.
template <int V>
__device__ __forceinline__ void to_codes(float (&v)[V], float inv, bool bad) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if (bad && (__float_as_uint(v[k]) & 0x7fffffffu) >= kInfBits) v[k] = __uint_as_float(0x7fffffffu);
        v[k] *= inv;
    }
}

// V codes as fp32 numbers (exact).
template <int V>
__device__ __forceinline__ void from_codes(const Raw<e4m3_t, V>& r, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = __half2float(__half(__nv_cvt_fp8_to_halfraw(r.w, __NV_E4M3)));
    } else {
        const __nv_fp8x2_storage_t* w = reinterpret_cast<const __nv_fp8x2_storage_t*>(&r.w);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(w[k], __NV_E4M3)));
            v[2 * k] = f.x;
            v[2 * k + 1] = f.y;
        }
    }
}

// Sums and maxima over the threads of a row: a warp, or the CTA (every thread of it calls; `part` has an entry per warp, and each
// warp combines them for itself, in one order).  Calls in a row alternate between two arrays: whoever writes one again is past
// a barrier that its readers reached after reading.
struct RowSums {
    float a, b, c;
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int N>
__device__ __forceinline__ void row_sums(RowSums& s, bool one_warp, float4* part) {
    s.a = warp_sum(s.a);
    if (N > 1) s.b = warp_sum(s.b);
    if (N > 2) s.c = warp_sum(s.c);
    if (one_warp) return;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = make_float4(s.a, s.b, s.c, 0.f);
    __syncthreads();
    const float4 q = lane < (int)(blockDim.x >> 5) ? part[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    s.a = warp_sum(q.x);
    if (N > 1) s.b = warp_sum(q.y);
    if (N > 2) s.c = warp_sum(q.z);
}
struct RowMaxima {
    uint32_t a, b;
};
__device__ __forceinline__ void row_sum_maxima(float& s, RowMaxima& m, bool one_warp, float4* part) {
    s = warp_sum(s);
    m.a = __reduce_max_sync(0xffffffffu, m.a);
    m.b = __reduce_max_sync(0xffffffffu, m.b);
    if (one_warp) return;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = make_float4(s, __uint_as_float(m.a), __uint_as_float(m.b), 0.f);
    __syncthreads();
    const float4 q = lane < (int)(blockDim.x >> 5) ? part[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    s = warp_sum(q.x);
    m.a = __reduce_max_sync(0xffffffffu, __float_as_uint(q.y));
    m.b = __reduce_max_sync(0xffffffffu, __float_as_uint(q.z));
}

// 1 / (1 + e^-z).  bf16 inputs: ex2.approx and rcp.approx, a few 2^-23 each, far inside the inputs' rounding; fp32 inputs:
// expf and a division.  z to -infinity gives 0, to infinity 1.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (sizeof(T) == 4) {
        return 1.f / (1.f + expf(-z));
    } else {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-z * kLog2e));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return r;
    }
}

// V weights from column e of a row (16-byte aligned with e where V > 1 and !SHIFTED), kept in the caches; those outside of
// [0, n) are 0.
template <int V, bool SHIFTED>
__device__ __forceinline__ void row_weights(const float* p, int e, int n, float (&w)[V]) {
    if constexpr (V == 1) {
        w[0] = __ldg(p + e);
    } else if constexpr (SHIFTED) {
#pragma unroll
        for (int k = 0; k < V; ++k) w[k] = e + k >= 0 && e + k < n ? __ldg(p + e + k) : 0.f;
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(p + e + k));
            w[k] = q.x;
            w[k + 1] = q.y;
            w[k + 2] = q.z;
            w[k + 3] = q.w;
        }
    }
}

}  // namespace ssd
