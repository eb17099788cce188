// Element access of the layer operators (sm_103a): V consecutive elements of a
// bf16, fp32 or e4m3 array moved as one access and widened to (or rounded from)
// fp32 in registers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace ssd {

typedef __nv_bfloat16 bf16_t;
typedef __nv_fp8_e4m3 e4m3_t;

template <int BYTES> struct Word;
template <> struct Word<1> { typedef uint8_t type; };
template <> struct Word<2> { typedef uint16_t type; };
template <> struct Word<4> { typedef uint32_t type; };
template <> struct Word<8> { typedef uint2 type; };
template <> struct Word<16> { typedef uint4 type; };
struct alignas(16) Word32B { uint4 lo, hi; };
template <> struct Word<32> { typedef Word32B type; };

// V elements of T as they lie in memory.  Loads are marked evict-first (each
// operand of these operators is read once) and stores streaming.
template <typename T, int V>
struct Raw {
    typedef typename Word<(int)sizeof(T) * V>::type W;
    W w;
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (sizeof(T) * V == 32) {
            w.lo = __ldcs(reinterpret_cast<const uint4*>(p));
            w.hi = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
        } else {
            w = __ldcs(reinterpret_cast<const W*>(p));
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (sizeof(T) * V == 32) {
            __stcs(reinterpret_cast<uint4*>(p), w.lo);
            __stcs(reinterpret_cast<uint4*>(p) + 1, w.hi);
        } else {
            __stcs(reinterpret_cast<W*>(p), w);
        }
    }
    // The first n of the V elements, one by one.
    __device__ __forceinline__ void load_some(const T* p, int n) {
        T* v = reinterpret_cast<T*>(&w);
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < n) v[k] = p[k];
    }
    // Those of the V elements from column e of a row that lie in its columns [0, n), one by one.
    __device__ __forceinline__ void store_within(T* row, int e, int n) const {
        const T* v = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (e + k >= 0 && e + k < n) row[e + k] = v[k];
    }
    __device__ __forceinline__ void zero() {
        if constexpr (sizeof(T) * V == 32) w.lo = w.hi = make_uint4(0, 0, 0, 0);
        else if constexpr (sizeof(T) * V == 16) w = make_uint4(0, 0, 0, 0);
        else if constexpr (sizeof(T) * V == 8) w = make_uint2(0, 0);
        else w = 0;
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
        const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (sizeof(T) == 2) v[k] = __bfloat162float(e[k]);
            else v[k] = e[k];
        }
    }
    __device__ __forceinline__ void set(const float (&v)[V]) {
        if constexpr (sizeof(T) == 4) {
            float* e = reinterpret_cast<float*>(&w);
#pragma unroll
            for (int k = 0; k < V; ++k) e[k] = v[k];
        } else if constexpr (sizeof(T) == 2) {
            if constexpr (V == 1) {
                const bf16_t b = __float2bfloat16_rn(v[0]);
                w = *reinterpret_cast<const uint16_t*>(&b);
            } else {
                __nv_bfloat162* e = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
                for (int k = 0; k < V / 2; ++k) e[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            }
        } else {
            // e4m3, round to nearest even, saturating; NaN stays NaN
            if constexpr (V == 1) {
                w = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
            } else {
                __nv_fp8x2_storage_t* e = reinterpret_cast<__nv_fp8x2_storage_t*>(&w);
#pragma unroll
                for (int k = 0; k < V / 2; ++k)
                    e[k] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * k], v[2 * k + 1]), __NV_SATFINITE, __NV_E4M3);
            }
        }
    }
};

// Larger of two values; NaN when either is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

}  // namespace ssd
