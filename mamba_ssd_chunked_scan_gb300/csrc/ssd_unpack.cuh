// What 8-bit rows stand for, by CTAs of the flat array (sm_103a): ssd_unpack_kernel's, and those of a launch that has other work too.
#pragma once
#include "ssd_kernels.h"
#include "ssd_rows.cuh"

namespace ssd {

constexpr int kFlat = 16, kFlatThreads = 256;   // elements per thread of the flat array, threads of a CTA

// Where codes' rows lie together and both arrays start on 16 bytes: a thread takes 16 elements of the flat array, of one unit or of
// several.  A CTA's first unit is divided out once, in 64 bits; the rest is in 32.
template <typename T>
__device__ __forceinline__ void unpack_flat(const PackArgs& a, unsigned cta) {
    const int64_t total = a.units * a.size, begin = (int64_t)cta * kFlatThreads * kFlat, at = begin + threadIdx.x * kFlat;
    if (at >= total) return;
    const int64_t unit0 = begin / a.size;
    const uint32_t n = a.size, k = (uint32_t)(begin - unit0 * a.size) + threadIdx.x * kFlat, over = k / n;
    uint32_t e = k - over * n;   // the first element's column in its unit
    const float* scales = a.scales + unit0 + over;
    const e4m3_t* codes = static_cast<const e4m3_t*>(a.codes) + at;
    T* out = static_cast<T*>(a.out) + at;
    const int count = total - at < kFlat ? (int)(total - at) : kFlat;
    Raw<e4m3_t, kFlat> q;
    q.zero();
    if (count == kFlat) q.load(codes);
    else q.load_some(codes, count);
    Two v[kFlat / 2];
    to_pairs(q, v);
    auto scale_at = [&](const float* p) { return a.power_only ? scale_power(__ldg(p)) : __ldg(p); };
    float s = scale_at(scales);
    if (e + kFlat <= n) {
#pragma unroll
        for (int j = 0; j < kFlat / 2; ++j) v[j] = v[j] * both(s);
    } else {
#pragma unroll
        for (int j = 0; j < kFlat; ++j) {
            if (e == n && j < count) {
                e = 0;
                s = scale_at(++scales);
            }
            ++e;
            if (j % 2) v[j / 2] = two(low(v[j / 2]), high(v[j / 2]) * s);
            else v[j / 2] = two(low(v[j / 2]) * s, high(v[j / 2]));
        }
    }
    constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
    for (int h = 0; h < kFlat / V; ++h) {
        Two p[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) p[j] = v[h * (V / 2) + j];
        Raw<T, V> o;
        from_pairs(p, o);
        if (h * V + V <= count) o.store(out + h * V);
        else o.store_within(out, h * V, count);
    }
}

}  // namespace ssd
