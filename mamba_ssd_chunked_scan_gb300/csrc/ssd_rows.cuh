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

// A scale as power * factor: a power of two of its sign, and a factor from 1 up to 2 (1 for zeros, subnormals, infinities and NaNs).
__device__ __forceinline__ float scale_factor(float s) {
    const uint32_t b = __float_as_uint(s), e = b >> 23 & 0xffu;
    return e > 0 && e < 255 ? __uint_as_float((b & 0x7fffffu) | 0x3f800000u) : 1.f;
}
__device__ __forceinline__ float scale_power(float s) {
    const uint32_t b = __float_as_uint(s), e = b >> 23 & 0xffu;
    return e > 0 && e < 255 ? __uint_as_float(b & 0xff800000u) : s;
}

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

// NaN in place of an infinity or a NaN.
__device__ __forceinline__ float nan_unless_finite(float v) {
    return (__float_as_uint(v) & 0x7fffffffu) >= kInfBits ? __uint_as_float(0x7fffffffu) : v;
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

// Two fp32 numbers in a register pair: one instruction does both (fma.rn.f32x2 and the like), and what these kernels run
// out of first is issue slots.
struct Two {
    uint64_t w;
};
__device__ __forceinline__ Two two(float lo, float hi) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.w) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ Two both(float v) { return two(v, v); }
__device__ __forceinline__ float low(Two a) { return __uint_as_float((uint32_t)a.w); }
__device__ __forceinline__ float high(Two a) { return __uint_as_float((uint32_t)(a.w >> 32)); }
__device__ __forceinline__ Two operator*(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.w) : "l"(a.w), "l"(b.w));
    return r;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.w) : "l"(a.w), "l"(b.w));
    return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.w) : "l"(a.w), "l"(b.w), "l"(c.w));
    return r;
}

// V elements as pairs, and back.
template <typename T, int V>
__device__ __forceinline__ void to_pairs(const Raw<T, V>& r, Two (&v)[V / 2]) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r.w);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) v[k] = two(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    } else {
        float f[V];
        if constexpr (sizeof(T) == 1) from_codes(r, f);
        else r.get(f);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) v[k] = two(f[2 * k], f[2 * k + 1]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void from_pairs(const Two (&v)[V / 2], Raw<T, V>& r) {
    float f[V];
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
        f[2 * k] = low(v[k]);
        f[2 * k + 1] = high(v[k]);
    }
    r.set(f);
}

// 1 / sqrt(x) by the special-function unit (relative error below 2^-22); 0 gives infinity.
__device__ __forceinline__ float rsqrt_of(float x) {
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One or two sums over the threads of a row: a warp, or the CTA of up to 32 warps (every thread of it calls, and adds the warps'
// sums for itself, in one order).  Two sums share their shuffles: at the first a lane passes on the one that it does not
// keep.  Calls in a row alternate between two arrays: whoever writes one again is past a barrier that its readers reached
// after reading.
struct RowPart {
    __align__(16) float sums[64];
    uint2 maxima[32];
};
// A warp's sums (of two, the second in lanes 16 to 31), and the CTA's from the warps'.
template <int N>
__device__ __forceinline__ float warp_sums(const float (&s)[N]) {
    constexpr uint32_t kAll = 0xffffffffu;
    float v = s[0];
    if constexpr (N == 2) {
        const bool up = threadIdx.x & 16;
        v = (up ? s[1] : s[0]) + __shfl_xor_sync(kAll, up ? s[0] : s[1], 16);
    }
#pragma unroll
    for (int o = N == 2 ? 8 : 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
template <int N>
__device__ __forceinline__ void leave_sums(float v, RowPart& part) {
    const int lane = threadIdx.x & 31;
    if (lane % (32 / N) == 0) part.sums[(threadIdx.x >> 5) * N + (N == 2 ? lane >> 4 : 0)] = v;
}
template <int N>
__device__ __forceinline__ void join_sums(float (&s)[N], const RowPart& part) {
    const int count = (blockDim.x >> 5) * N;
    Two t = both(0.f), u = t;
    int k = 0;
#pragma unroll 4
    for (; k + 4 <= count; k += 4) {
        const float4 q = *reinterpret_cast<const float4*>(part.sums + k);
        t = t + two(q.x, q.y);
        u = u + two(q.z, q.w);
    }
    if (k < count) {   // what is left
        t = t + two(part.sums[k], k + 1 < count ? part.sums[k + 1] : 0.f);
        if (k + 2 < count) u = u + two(part.sums[k + 2], 0.f);
    }
    t = t + u;
    if constexpr (N == 1) {
        s[0] = low(t) + high(t);
    } else {
        s[0] = low(t);
        s[1] = high(t);
    }
}
template <int N>
__device__ __forceinline__ void row_sums(float (&s)[N], bool one_warp, RowPart& part) {
    static_assert(N == 1 || N == 2, "");
    const float v = warp_sums(s);
    if (one_warp) {
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] = N == 1 ? v : __shfl_sync(0xffffffffu, v, 16 * k);
        return;
    }
    leave_sums<N>(v, part);
    __syncthreads();
    join_sums(s, part);
}

// The lanes of a warp that share a row with this one: LANES of them side by side, a power of two (0: all).
template <int LANES>
__device__ __forceinline__ uint32_t row_mask() {
    return LANES % 32 == 0 ? 0xffffffffu : ((1u << (LANES % 32)) - 1) << (threadIdx.x & (32 - LANES));
}
// Two sums over them.
template <int LANES>
__device__ __forceinline__ void lane_sums(float (&s)[2]) {
    const uint32_t mask = row_mask<LANES>();
    const bool up = threadIdx.x & (LANES / 2);
    float v = (up ? s[1] : s[0]) + __shfl_xor_sync(mask, up ? s[0] : s[1], LANES / 2);
#pragma unroll
    for (int o = LANES / 4; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    s[0] = __shfl_sync(mask, v, 0, LANES);
    s[1] = __shfl_sync(mask, v, LANES / 2, LANES);
}

// A sum and two maxima over the threads of a row: LANES lanes of a warp, or (0) the CTA, by one barrier.
struct RowMaxima {
    uint32_t a, b;
};
template <int LANES>
__device__ __forceinline__ void row_sum(float (&s)[1], RowPart& part) {
    if constexpr (LANES == 0) {
        row_sums(s, false, part);
    } else {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) s[0] += __shfl_xor_sync(row_mask<LANES>(), s[0], o);
    }
}
template <int LANES>
__device__ __forceinline__ uint32_t row_maximum(uint32_t m, uint32_t (&part)[32]) {
    m = __reduce_max_sync(row_mask<LANES>(), m);
    if constexpr (LANES == 0) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, lane < (int)(blockDim.x >> 5) ? part[lane] : 0u);
    }
    return m;
}
// The sum is the same as row_sum's.
template <int LANES>
__device__ __forceinline__ void row_sum_maxima(float (&s)[1], RowMaxima& m, RowPart& part) {
    m.a = __reduce_max_sync(row_mask<LANES>(), m.a);
    m.b = __reduce_max_sync(row_mask<LANES>(), m.b);
    if constexpr (LANES != 0) {
        row_sum<LANES>(s, part);
    } else {
        const float v = warp_sums(s);
        const int lane = threadIdx.x & 31;
        leave_sums<1>(v, part);
        if (lane == 0) part.maxima[threadIdx.x >> 5] = make_uint2(m.a, m.b);
        __syncthreads();
        join_sums(s, part);
        const uint2 q = lane < (int)(blockDim.x >> 5) ? part.maxima[lane] : make_uint2(0, 0);
        m.a = __reduce_max_sync(0xffffffffu, q.x);
        m.b = __reduce_max_sync(0xffffffffu, q.y);
    }
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

template <typename T>
__device__ __forceinline__ Two sigmoid(Two z) {
    if constexpr (sizeof(T) == 4) {
        return two(sigmoid<T>(low(z)), sigmoid<T>(high(z)));
    } else {
        const Two t = z * both(-kLog2e);
        float e, f;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(low(t)));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(high(t)));
        const Two q = two(e, f) + both(1.f);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(low(q)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(high(q)));
        return two(e, f);
    }
}

// A thread's part of a row, E elements: vectors of V (16 bytes of the row's type), vector c from column column(c) on; or (V = 2)
// pairs of single elements, columns e and e + nt, whatever the alignment.  SHIFTED: see ssd_ring.cuh; `left`: columns to the
// arrays' end from the row's start.
template <int V, bool SHIFTED>
struct Place {
    int tid, nt, shift, n;
    int64_t left;
    __device__ __forceinline__ int column(int c) const { return V > 2 ? (tid + c * nt) * V - shift : tid + 2 * c * nt; }
};
template <typename K, int V, int E, bool SHIFTED>
struct Part {
    static constexpr int kEach = V > 2 ? V : 1, C = E / V;
    Raw<K, kEach> q[E / kEach];
    // `row`: the row's column 0
    __device__ __forceinline__ void load(const K* row, const Place<V, SHIFTED>& p) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = p.column(c);
            if constexpr (V > 2) {
                q[c].zero();
                if (e < p.n) {
                    if (!SHIFTED || e + V <= p.left) q[c].load(row + e);
                    else q[c].load_some(row + e, (int)(p.left - e));
                    if (SHIFTED && (e < 0 || e + V > p.n)) {   // a neighbour's elements
                        K* v = reinterpret_cast<K*>(&q[c].w);
                        Raw<K, 1> none;
                        none.zero();
#pragma unroll
                        for (int k = 0; k < V; ++k)
                            if (e + k < 0 || e + k >= p.n) v[k] = *reinterpret_cast<K*>(&none.w);
                    }
                }
            } else {
                q[2 * c].zero();
                q[2 * c + 1].zero();
                if (e < p.n) q[2 * c].load(row + e);
                if (e + p.nt < p.n) q[2 * c + 1].load(row + e + p.nt);
            }
        }
    }
    __device__ __forceinline__ void store(K* row, const Place<V, SHIFTED>& p, int c) const {
        const int e = p.column(c);
        if constexpr (V > 2) {
            if (SHIFTED && (e < 0 || e + V > p.n)) q[c].store_within(row, e, p.n);
            else if (e < p.n) q[c].store(row + e);
        } else {
            if (e < p.n) q[2 * c].store(row + e);
            if (e + p.nt < p.n) q[2 * c + 1].store(row + e + p.nt);
        }
    }
    __device__ __forceinline__ void get(int c, Two (&v)[V / 2]) const {
        if constexpr (V > 2) {
            to_pairs(q[c], v);
        } else {
            float f[1], g[1];
            q[2 * c].get(f);
            q[2 * c + 1].get(g);
            v[0] = two(f[0], g[0]);
        }
    }
    __device__ __forceinline__ void set(int c, const Two (&v)[V / 2]) {
        if constexpr (V > 2) {
            from_pairs(v, q[c]);
        } else {
            const float f[1] = {low(v[0])}, g[1] = {high(v[0])};
            q[2 * c].set(f);
            q[2 * c + 1].set(g);
        }
    }
    // largest magnitude; and over finite elements alone
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < E / kEach; ++c) m = max(m, magnitude(q[c]));
        return m;
    }
    __device__ __forceinline__ uint32_t finite_top() const {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < E / kEach; ++c) m = max(m, finite_magnitude(q[c]));
        return m;
    }
};
// Vector c of a row times `inv` as codes; `bad`: some element of the row is infinite or NaN.
template <int V, int E, bool SHIFTED>
__device__ __forceinline__ void store_codes(e4m3_t* row, const Place<V, SHIFTED>& p, int c, Two (&v)[V / 2], float inv, bool bad) {
    if (bad) {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) v[k] = two(nan_unless_finite(low(v[k])), nan_unless_finite(high(v[k])));
    }
#pragma unroll
    for (int k = 0; k < V / 2; ++k) v[k] = v[k] * both(inv);
    Part<e4m3_t, V, E, SHIFTED> q;
    q.set(c, v);
    q.store(row, p, c);
}
// Pair c of a row's weights, kept in the caches; 0 outside of the row.
__device__ __forceinline__ Two pair_weights(const float* p, const Place<2, false>& at, int c) {
    const int e = at.column(c);
    return two(e < at.n ? __ldg(p + e) : 0.f, e + at.nt < at.n ? __ldg(p + e + at.nt) : 0.f);
}

// V weights from column e of a row (16-byte aligned with e where !SHIFTED), kept in the caches; those outside of
// [0, n) are 0.
template <int V, bool SHIFTED>
__device__ __forceinline__ void row_weights(const float* p, int e, int n, float (&w)[V]) {
    if constexpr (SHIFTED) {
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
