// The kernels of ssd_block_norm_bwd.cu, which has the formulas; its instances are spread over several files so that they compile
// side by side.
#pragma once
#include <atomic>

#include "ssd_kernels.h"
#include "ssd_ring.cuh"

namespace ssd {

constexpr int kMaxStages = 4;

// Threads per SM that the registers of E elements a thread allow.
constexpr int threads_sm(int elems, bool res) { return elems == kNarrowElems || !res ? 640 : 512; }

constexpr int loose_threads_sm(int elems) { return elems == kNarrowElems ? 640 : 512; }   // where no vectors fit

// A warp's record of one row: its lanes' vectors of each operand, piece by piece (16 bytes a lane, then codes, then scales), so that
// whole lines arrive in one place and every offset is a constant (records of a thread each, 112 bytes apart, took the copies from 5.5
// to 3.6 TB/s).  Offsets here are a lane's bytes before a piece: 32 times that in the record.
template <typename T, typename R, int E, bool GATE, bool RES, bool XP, bool HP>
struct Record {
    static constexpr int kVec = 16 / (int)sizeof(T);
    static constexpr int t = E * (int)sizeof(T), r = E * (int)sizeof(R);   // bytes of an operand of these types; of codes E
    static constexpr int dout = 0;
    static constexpr int dres = dout + t;
    static constexpr int h = dres + (RES ? r : 0);
    static constexpr int x = h + (RES && !HP ? r : 0);
    static constexpr int xs = RES ? 2 : 1;   // of x two rows' where the record is one row's otherwise
    static constexpr int gate = x + (XP ? 0 : xs * t);
    static constexpr int codes = gate + (GATE && !XP ? t : 0);
    static constexpr int x_codes = codes, gate_codes = x_codes + (XP ? xs * E : 0), h_codes = gate_codes + (XP && GATE ? E : 0);
    static constexpr int x_scale = h_codes + (RES && HP ? E : 0);
    static constexpr int gate_scale = x_scale + (XP ? 4 : 0), h_scale = gate_scale + (XP && GATE ? 4 : 0);
    static constexpr int bytes = h_scale + (RES && HP ? 4 : 0);
    static constexpr int weight = E * 4, weights = (RES ? 2 : 1) * weight;   // the weights' record
};

// silu's slope s + silu (1 - s), of s = 1 / (1 + e^-z) and silu = z s.  Where s is 1 so is the slope, however large z is (as
// s (1 - silu) + silu it is 0 or 2 from z = 2^24 on, where 1 - silu is rounded).
__device__ __forceinline__ Two silu_slope(Two s, Two silu) { return fma(silu, fma(s, both(-1.f), both(1.f)), s); }
// silu(z) and its slope.
template <typename T>
__device__ __forceinline__ void silu(Two z, Two& value, Two& slope) {
    const Two s = sigmoid<T>(z);
    value = z * s;
    slope = silu_slope(s, value);
}

// A slot's rows: place.row, place.row + place.step, ... before place.end, one group of each; and the row of shares that it leaves.
struct Slot {
    int group, row, end, step, share;
};
__device__ __forceinline__ Slot slot_of(const BlockNormBwdArgs& a, int id) {
    const bool late = id >= a.slots;
    const int k = late ? id - a.slots : id, line = k / a.groups;
    Slot s;
    s.group = k - line * a.groups;
    s.row = late ? a.early_rows + line : line;
    s.end = late ? (int)a.rows : a.early_rows;
    s.step = (late ? a.late_slots : a.slots) / a.groups;
    s.share = late ? a.slots / a.groups + line : line;
    return s;
}

// LANES: lanes of a warp that take a row (a slot); 0: a CTA does, and where its rows lie is the same number for all of its
// threads (uniform registers hold it).  XP: x (and gate) are codes; HP: h is.  SHIFTED: see ssd_ring.cuh.
template <typename T, typename R, int E, int LANES, bool SHIFTED, bool GATE, bool RES, bool XP, bool HP>
__global__ void __launch_bounds__(threads_sm(E, RES)) ssd_block_norm_bwd_kernel(const __grid_constant__ BlockNormBwdArgs a) {
    typedef Record<T, R, E, GATE, RES, XP, HP> Rec;
    typedef typename Pick<XP, e4m3_t, T>::type X;
    typedef typename Pick<HP, e4m3_t, R>::type H;
    constexpr bool kCta = LANES == 0;
    // With a residual silu and its slope stay in registers from one pass to the next, and all of a record but x is free for the next
    // row before the last pass: one stage is enough then, which leaves room for three CTAs instead of two, and a second place for x.
    constexpr bool kKeep = RES, kEarly = RES;
    constexpr bool kPairs = RES && sizeof(R) > sizeof(T);   // lanes copy for their neighbours
    const uint32_t mask = row_mask<LANES>();
    constexpr int V = Rec::kVec, C = E / V, P = V / 2;
    // the operands' first pieces
    constexpr int kD = 32 * Rec::dout, kR = 32 * Rec::dres, kX = 32 * (XP ? Rec::x_codes : Rec::x), kZ = 32 * (XP ? Rec::gate_codes : Rec::gate),
                  kH = 32 * (HP ? Rec::h_codes : Rec::h), kStage = 32 * Rec::bytes, kXs = 32 * E * (int)sizeof(X);
    __shared__ RowPart part[2];
    extern __shared__ __align__(16) unsigned char ring[];
    const int tid = kCta ? threadIdx.x : threadIdx.x % (kCta ? 32 : LANES), nt = kCta ? blockDim.x : LANES;
    const int id = kCta ? blockIdx.x : blockIdx.x * a.slots_per_cta + threadIdx.x / (kCta ? 32 : LANES);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();
    pdl_wait();
    if (!kCta && id >= a.slots + a.late_slots) return;
    const int n = a.size;
    const Slot place = slot_of(a, id);
    const int group = place.group, first = group * n, step = place.step;   // the group's first column
    const uint32_t line = place.row;                                       // the slot's first row
    const bool next = RES && a.dout;
    const uint32_t my_units = (uint32_t)place.end * a.groups, unit_step = (uint32_t)step * a.groups,
                   unit0 = line * a.groups + group;
    const int shift = SHIFTED ? (int)((uint64_t)unit0 * n % V) : 0;
    const int e0 = tid * V - shift, span = nt * V;   // first column of the thread's vector 0; columns from one vector to the next
    // a warp's shared memory: its lanes' weights, then the stages
    unsigned char* const wrec = ring + warp * (32 * Rec::weights + a.stages * kStage);
    unsigned char* const rec0 = wrec + 32 * Rec::weights;
    // the weights' record; and zeros for vectors past the row's end, which nothing is copied into
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = e0 + c * span;
        float w[V] = {}, w2[V] = {};
        if (e < n) {
            row_weights<V, SHIFTED>(a.weight + first, e, n, w);
            if (next) row_weights<V, SHIFTED>(a.next_weight, e, n, w2);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            reinterpret_cast<float*>(wrec + piece<float, V>(c, k / 4, lane))[k % 4] = w[k];
            if (RES) reinterpret_cast<float*>(wrec + 32 * Rec::weight + piece<float, V>(c, k / 4, lane))[k % 4] = w2[k];
        }
        if (e >= n) {
            for (int s = 0; s < a.stages; ++s) {
                unsigned char* r = rec0 + s * kStage;
                clear_head<T, V>(r + kD, c, lane, V);
                for (int k = 0; k < Rec::xs; ++k) clear_head<X, V>(r + kX + k * kXs, c, lane, V);
                if (GATE) clear_head<X, V>(r + kZ, c, lane, V);
                if (RES) clear_head<H, V>(r + kH, c, lane, V);
                if (RES) clear_head<R, V>(r + kR, c, lane, V);
            }
        }
    }
    auto weight = [&](int c, Two (&w)[P]) { to_pairs(piece_vector<float, V>(wrec, c, lane), w); };
    auto next_weight = [&](int c, Two (&w)[P]) { to_pairs(piece_vector<float, V>(wrec + 32 * Rec::weight, c, lane), w); };
    // Where vector 0 of thread 0 lies in each operand of the next row to ask for, in each result of the row at hand, and how far it
    // is from one of the slot's rows to the next (in elements).
    const int64_t at0 = (int64_t)unit0 * n - shift, gate0 = (int64_t)line * a.gate_stride + first - shift;
    const int64_t far = (int64_t)unit_step * n, gate_far = (int64_t)step * a.gate_stride;
    auto in = [](const void* p, int64_t elems, int size) { return static_cast<const unsigned char*>(p) + elems * size; };
    const unsigned char *p_dout = in(a.dout, at0, sizeof(T)), *p_x = in(a.x, at0, sizeof(X)), *p_gate = in(a.gate, gate0, sizeof(X)),
                        *p_h = in(a.h, at0, sizeof(H)), *p_dres = in(a.dres, at0, sizeof(R));
    auto out = [](void* p, int64_t elems, int size) { return static_cast<unsigned char*>(p) + elems * size; };
    unsigned char *q_dx = out(a.dx, at0, sizeof(T)), *q_dres = out(a.dres_out, at0, sizeof(R)), *q_out = out(a.out, at0, sizeof(T)),
                  *q_dgate = out(a.dgate, (int64_t)line * a.dgate_stride + first - shift, sizeof(T));
    uint32_t unit_ask = unit0;
    // Ask for the next row, into a stage; x into its place at `x_at`.
    auto ask_row = [&](int stage, int x_at) {
        if (unit_ask < my_units) {
            const uint32_t to = (uint32_t)__cvta_generic_to_shared(rec0) + stage * kStage;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = e0 + c * span;
                const uint32_t t = (uint32_t)tid * V;
                const int64_t s = c * span;
                if (!RES || next) ask<T, V, SHIFTED>(to + kD, c, lane, p_dout + s * sizeof(T), t * sizeof(T), e, n);
                if (next) ask<H, V, SHIFTED>(to + kH, c, lane, p_h + s * sizeof(H), t * sizeof(H), e, n);
                if (RES) ask<R, V, SHIFTED>(to + kR, c, lane, p_dres + s * sizeof(R), t * sizeof(R), e, n);
                if (GATE) ask<X, V, SHIFTED>(to + kZ, c, lane, p_gate + s * sizeof(X), t * sizeof(X), e, n);
                ask<X, V, SHIFTED>(to + kX + x_at, c, lane, p_x + s * sizeof(X), t * sizeof(X), e, n);
            }
            if (XP) copy_async<4>(to + 32 * Rec::x_scale + 4 * lane, a.x_scales + unit_ask, 4);
            if (XP && GATE) copy_async<4>(to + 32 * Rec::gate_scale + 4 * lane, a.gate_scales + unit_ask, 4);
            if (HP && next) copy_async<4>(to + 32 * Rec::h_scale + 4 * lane, a.h_scales + unit_ask, 4);
            if (!RES || next) p_dout += far * sizeof(T);
            if (GATE) p_gate += gate_far * sizeof(X);
            if (next) p_h += far * sizeof(H);
            if (RES) p_dres += far * sizeof(R);
            p_x += far * sizeof(X);
            unit_ask += unit_step;
        }
        copies_commit();
    };
    auto sums = [&](float (&s)[2], int turn) {
        if constexpr (kCta) row_sums(s, false, part[turn]);
        else lane_sums<LANES>(s);
    };
    Two dw[C][P], dn[RES ? C : 1][P];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < P; ++k) {
            dw[c][k] = both(0.f);
            if (RES) dn[c][k] = both(0.f);
        }
    for (int s = 0; s < (kEarly ? 1 : a.stages - 1); ++s) ask_row(s, 0);
    int stage = 0, turn = 0, x_at = 0;
    for (uint32_t unit = unit0; unit < my_units; unit += unit_step) {
        unsigned char* const rec = rec0 + stage * kStage;
        if constexpr (!kEarly) {
            ask_row(stage > 0 ? stage - 1 : a.stages - 1, 0);   // where the row before lay
            if (++stage == a.stages) stage = 0;
        }
        copies_wait(kEarly ? 0 : a.stages - 1);
        if constexpr (kPairs) __syncwarp(mask);
        if (SHIFTED && e0 < 0) {
            if (!RES || next) clear_head<T, V>(rec + kD, 0, lane, shift);
            clear_head<X, V>(rec + kX + x_at, 0, lane, shift);
            if (GATE) clear_head<X, V>(rec + kZ, 0, lane, shift);
            if (next) clear_head<H, V>(rec + kH, 0, lane, shift);
            if (RES) clear_head<R, V>(rec + kR, 0, lane, shift);
        }
        // codes of x and h stay codes; their scales join the sums' and the row's factors
        float xs = 1.f, gs = 1.f, hs = 1.f;
        if (XP) xs = *reinterpret_cast<const float*>(rec + 32 * Rec::x_scale + 4 * lane);
        if (XP && GATE) gs = *reinterpret_cast<const float*>(rec + 32 * Rec::gate_scale + 4 * lane);
        if (HP && next) hs = *reinterpret_cast<const float*>(rec + 32 * Rec::h_scale + 4 * lane);
        auto dout_of = [&](int c, Two (&v)[P]) { to_pairs(piece_vector<T, V>(rec + kD, c, lane), v); };
        const unsigned char* const rec_x = rec + kX + x_at;
        auto x_of = [&](int c, Two (&v)[P]) { to_pairs(piece_vector<X, V>(rec_x, c, lane), v); };
        auto gate_of = [&](int c, Two (&v)[P]) {
            to_pairs(piece_vector<X, V>(rec + kZ, c, lane), v);
            if constexpr (XP) {
#pragma unroll
                for (int k = 0; k < P; ++k) v[k] = v[k] * both(gs);
            }
        };
        auto h_of = [&](int c, Two (&v)[P]) { to_pairs(piece_vector<H, V>(rec + kH, c, lane), v); };
        const uint32_t t = (uint32_t)tid * V;
        // What is kept of a row beside its record: the gate's sigmoid (or silu and its slope), and the gradient of u rstd1 weight.
        Two sg[GATE ? C : 1][P], sl[GATE && kKeep ? C : 1][P], g1[RES ? C : 1][P];
        Two r2 = both(0.f), r2h = r2, k2 = r2;
        if constexpr (RES) {
            if (next) {
                Two hh = both(0.f), ph = hh;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    Two h[P], d[P], w[P];
                    h_of(c, h);
                    dout_of(c, d);
                    next_weight(c, w);
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        hh = fma(h[k], h[k], hh);
                        ph = fma(d[k] * w[k], h[k], ph);
                    }
                }
                float s[2] = {low(hh) + high(hh), low(ph) + high(ph)};
                sums(s, turn);
                turn ^= 1;
                if (HP) {   // not hs * hs, which may be 0 or infinite
                    s[0] = s[0] * hs * hs;
                    s[1] *= hs;
                }
                const float rstd2 = rsqrt_of(s[0] * a.inv_size + a.eps);
                r2 = both(rstd2);
                r2h = both(HP ? rstd2 * hs : rstd2);
                const float k = -(s[1] * rstd2 * rstd2 * a.inv_size) * rstd2;   // h times it: -rstd2 hh mean(p2 hh)
                k2 = both(HP ? k * hs : k);
            }
        }
        Two uu = both(0.f), pu = uu;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Two x[P], w[P], g[P];
            if constexpr (RES) {
                to_pairs(piece_vector<R, V>(rec + kR, c, lane), g);
                if (next) {
                    Two h[P], d[P];
                    h_of(c, h);
                    dout_of(c, d);
                    next_weight(c, w);
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        g[k] = fma(d[k], w[k] * r2, fma(h[k], k2, g[k]));
                        dn[c][k] = fma(d[k], h[k] * r2h, dn[c][k]);
                    }
                }
                put<R, V, SHIFTED>(q_dres + c * span * (int64_t)sizeof(R), t * sizeof(R), e0 + c * span, n, mask, g);
#pragma unroll
                for (int k = 0; k < P; ++k) g1[c][k] = g[k] = both(a.scale) * g[k];
            } else {
                dout_of(c, g);
            }
            x_of(c, x);
            weight(c, w);
            if constexpr (GATE) {
                Two z[P];
                gate_of(c, z);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    if constexpr (kKeep) {
                        silu<T>(z[k], sg[c][k], sl[c][k]);
                        if (XP) sl[c][k] = sl[c][k] * both(xs);
                        x[k] = x[k] * sg[c][k];
                    } else {
                        sg[c][k] = sigmoid<T>(z[k]);
                        x[k] = x[k] * (z[k] * sg[c][k]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < P; ++k) {
                uu = fma(x[k], x[k], uu);
                pu = fma(g[k] * w[k], x[k], pu);
            }
        }
        if constexpr (kPairs) __syncwarp(mask);
        if constexpr (kEarly) {   // this row needs no more than x
            x_at ^= kXs;
            ask_row(0, x_at);
        }
        float s[2] = {low(uu) + high(uu), low(pu) + high(pu)};
        if (XP) {   // a thread's sums already: codes are up to 448, and all of a row's times large gates may pass fp32's range
            s[0] = s[0] * xs * xs;
            s[1] *= xs;
        }
        sums(s, turn);
        turn ^= 1;
        const float rstd = rsqrt_of(s[0] * a.inv_size + a.eps), mean = -(s[1] * a.inv_size * rstd * rstd) * rstd;
        const Two r1 = both(rstd), r1x = both(XP ? rstd * xs : rstd), k1 = both(XP ? mean * xs : mean);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Two w[P], g[P], x[P], z[P], du[P], o[P];
            const int e = e0 + c * span;
            weight(c, w);
            x_of(c, x);
            if constexpr (!RES) dout_of(c, g);
            if constexpr (GATE && !kKeep) gate_of(c, z);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                if constexpr (GATE) z[k] = kKeep ? sg[c][k] : z[k] * sg[c][k];   // silu
                if constexpr (RES) g[k] = g1[c][k];
                const Two u = GATE ? x[k] * z[k] : x[k];
                o[k] = u * r1x;
                du[k] = fma(g[k] * w[k], r1, u * k1);
                dw[c][k] = fma(g[k], o[k], dw[c][k]);
            }
            if (!RES && a.out) {
#pragma unroll
                for (int k = 0; k < P; ++k) o[k] = o[k] * w[k];
                put<T, V, SHIFTED>(q_out + c * span * (int64_t)sizeof(T), t * sizeof(T), e, n, mask, o);
            }
            if constexpr (GATE) {
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const Two slope = kKeep ? sl[c][k] : silu_slope(sg[c][k], z[k]);
                    o[k] = du[k] * (x[k] * slope);
                    if (XP && !kKeep) o[k] = o[k] * both(xs);
                    du[k] = du[k] * z[k];
                }
                put<T, V, SHIFTED>(q_dgate + c * span * (int64_t)sizeof(T), t * sizeof(T), e, n, mask, o);
            }
            put<T, V, SHIFTED>(q_dx + c * span * (int64_t)sizeof(T), t * sizeof(T), e, n, mask, du);
        }
        q_dx += far * sizeof(T);
        if (GATE) q_dgate += (int64_t)step * a.dgate_stride * (int64_t)sizeof(T);
        if (RES) q_dres += far * sizeof(R);
        if (!RES) q_out += far * sizeof(T);
    }
    const int width = n * a.groups, columns = RES && a.next_weight ? 2 * width : width;
    float* share = a.shares + (int64_t)place.share * columns + first;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = e0 + c * span;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (e + k < 0 || e + k >= n) continue;
            share[e + k] = k % 2 ? high(dw[c][k / 2]) : low(dw[c][k / 2]);
            if (RES && a.next_weight) share[width + e + k] = k % 2 ? high(dn[c][k / 2]) : low(dn[c][k / 2]);
        }
    }
}

// A thread's elements of a row for operands that no vectors fit: columns tid, tid + nt, ..., as they lie in memory.
template <typename K, int E>
struct Loose {
    Raw<K, 1> q[E];
    __device__ __forceinline__ void load(const void* p, int64_t at, int tid, int nt, int n) {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            q[k].zero();
            if (tid + k * nt < n) q[k].load(static_cast<const K*>(p) + at + tid + k * nt);
        }
    }
    __device__ __forceinline__ Two get(int c) const {
        float f[1], g[1];
        if constexpr (sizeof(K) == 1) {
            from_codes(q[2 * c], f);
            from_codes(q[2 * c + 1], g);
        } else {
            q[2 * c].get(f);
            q[2 * c + 1].get(g);
        }
        return two(f[0], g[0]);
    }
};
// Of type K, or codes times the row's scale (these are one byte of each element's 16 or 32 bits).
template <typename K, int E>
struct Either {
    Loose<K, E> plain;
    __device__ __forceinline__ void load(const void* p, bool packed, int64_t at, int tid, int nt, int n) {
        if (packed) {
            Loose<e4m3_t, E> codes;
            codes.load(p, at, tid, nt, n);
#pragma unroll
            for (int k = 0; k < E; ++k) plain.q[k].w = codes.q[k].w;
        } else {
            plain.load(p, at, tid, nt, n);
        }
    }
    __device__ __forceinline__ Two get(bool packed, Two scale, int c) const {
        if (!packed) return plain.get(c);
        float f[1], g[1];
        Raw<e4m3_t, 1> q;
        q.w = (uint8_t)plain.q[2 * c].w;
        from_codes(q, f);
        q.w = (uint8_t)plain.q[2 * c + 1].w;
        from_codes(q, g);
        return two(f[0], g[0]) * scale;
    }
};
template <typename K>
__device__ __forceinline__ void put_loose(K* row, int c, int tid, int nt, int n, Two v) {
    Raw<K, 1> q;
    const float f[1] = {low(v)}, g[1] = {high(v)};
    const int e = tid + 2 * c * nt;
    q.set(f);
    if (e < n) q.store(row + e);
    q.set(g);
    if (e + nt < n) q.store(row + e + nt);
}

// The same for rows and operands that no vectors fit: single elements, all of a row's asked for before the first is used.
template <typename T, typename R, int E, bool GATE, bool RES>
__global__ void __launch_bounds__(loose_threads_sm(E)) ssd_block_norm_bwd_loose(const __grid_constant__ BlockNormBwdArgs a) {
    constexpr int C = E / 2;
    __shared__ RowPart part[2];
    const bool one_warp = a.slots_per_cta > 1 || blockDim.x == 32;
    const int slot = one_warp ? threadIdx.x >> 5 : 0;
    const int tid = one_warp ? threadIdx.x & 31 : threadIdx.x;
    const int nt = one_warp ? 32 : blockDim.x;
    const int id = blockIdx.x * a.slots_per_cta + slot;
    pdl_trigger();
    pdl_wait();
    if (id >= a.slots + a.late_slots) return;   // whole warps of a many-slot CTA, which has no barrier
    const int n = a.size;
    const Slot place = slot_of(a, id);
    const int group = place.group, first = group * n, step = place.step;
    const bool next = RES && a.dout;
    Two dw[C], dn[RES ? C : 1];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        dw[c] = both(0.f);
        if (RES) dn[c] = both(0.f);
    }
    auto weights = [&](const float* p, int c) {
        const int e = tid + 2 * c * nt;
        return two(e < n ? __ldg(p + e) : 0.f, e + nt < n ? __ldg(p + e + nt) : 0.f);
    };
    int turn = 0;
    for (uint32_t row = place.row; row < (uint32_t)place.end; row += step) {
        const uint32_t unit = row * a.groups + group;
        const int64_t at = (int64_t)unit * n;
        Loose<T, E> dq;
        Either<T, E> xq, zq;
        Either<R, E> hq;
        Loose<R, E> rq;
        xq.load(a.x, a.x_scales, at, tid, nt, n);
        if (GATE) zq.load(a.gate, a.gate_scales, (int64_t)row * a.gate_stride + first, tid, nt, n);
        if (!RES || next) dq.load(a.dout, at, tid, nt, n);
        if (next) hq.load(a.h, a.h_scales, at, tid, nt, n);
        if (RES) rq.load(a.dres, at, tid, nt, n);
        const Two xs = both(a.x_scales ? __ldg(a.x_scales + unit) : 1.f);
        const Two gs = both(GATE && a.gate_scales ? __ldg(a.gate_scales + unit) : 1.f);
        const Two hs = both(next && a.h_scales ? __ldg(a.h_scales + unit) : 1.f);
        Two sg[GATE ? C : 1], g1[RES ? C : 1];
        Two r2 = both(0.f), k2 = r2;
        if constexpr (RES) {
            if (next) {
                Two hh = both(0.f), ph = hh;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const Two h = hq.get(a.h_scales, hs, c);
                    hh = fma(h, h, hh);
                    ph = fma(dq.get(c) * weights(a.next_weight, c), h, ph);
                }
                float s[2] = {low(hh) + high(hh), low(ph) + high(ph)};
                row_sums(s, one_warp, part[turn]);
                turn ^= 1;
                const float rstd2 = rsqrt_of(s[0] * a.inv_size + a.eps);
                r2 = both(rstd2);
                k2 = both(-(s[1] * rstd2 * rstd2 * a.inv_size) * rstd2);
            }
        }
        Two uu = both(0.f), pu = uu;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Two g;
            if constexpr (RES) {
                g = rq.get(c);
                if (next) {
                    const Two h = hq.get(a.h_scales, hs, c), d = dq.get(c);
                    g = fma(d, weights(a.next_weight, c) * r2, fma(h, k2, g));
                    dn[c] = fma(d, h * r2, dn[c]);
                }
                put_loose(static_cast<R*>(a.dres_out) + at, c, tid, nt, n, g);
                g1[c] = g = both(a.scale) * g;
            } else {
                g = dq.get(c);
            }
            Two u = xq.get(a.x_scales, xs, c);
            if constexpr (GATE) {
                const Two z = zq.get(a.gate_scales, gs, c);
                sg[c] = sigmoid<T>(z);
                u = u * (z * sg[c]);
            }
            uu = fma(u, u, uu);
            pu = fma(g * weights(a.weight + first, c), u, pu);
        }
        float s[2] = {low(uu) + high(uu), low(pu) + high(pu)};
        row_sums(s, one_warp, part[turn]);
        turn ^= 1;
        const float rstd = rsqrt_of(s[0] * a.inv_size + a.eps);
        const Two r1 = both(rstd), k1 = both(-(s[1] * a.inv_size * rstd * rstd) * rstd);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Two g, z;
            if constexpr (RES) g = g1[c];
            else g = dq.get(c);
            const Two x = xq.get(a.x_scales, xs, c), w = weights(a.weight + first, c);
            Two u = x;
            if constexpr (GATE) {
                z = zq.get(a.gate_scales, gs, c) * sg[c];
                u = x * z;
            }
            const Two o = u * r1;
            Two du = fma(g * w, r1, u * k1);
            dw[c] = fma(g, o, dw[c]);
            if (!RES && a.out) put_loose(static_cast<T*>(a.out) + at, c, tid, nt, n, o * w);
            if constexpr (GATE) {
                put_loose(static_cast<T*>(a.dgate) + (int64_t)row * a.dgate_stride + first, c, tid, nt, n,
                          du * (x * silu_slope(sg[c], z)));
                du = du * z;
            }
            put_loose(static_cast<T*>(a.dx) + at, c, tid, nt, n, du);
        }
    }
    const int width = n * a.groups, columns = RES && a.next_weight ? 2 * width : width;
    float* share = a.shares + (int64_t)place.share * columns + first;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = tid + (2 * c + k) * nt;
            if (e >= n) continue;
            share[e] = k ? high(dw[c]) : low(dw[c]);
            if (RES && a.next_weight) share[width + e] = k ? high(dn[c]) : low(dn[c]);
        }
}

// How a call's rows are spread: a slot's lanes (0: a CTA), threads of a CTA, its slots, and all slots (a number of rows at a time, each
// of its groups).
struct RowPlan {
    int elems, lanes, threads, slots_per_cta, slots, late_slots, early_rows, grid;
};

// Threads of a CTA that takes rows by itself, and CTAs that the registers of so many threads an SM hold.
inline int row_threads(int span, int elems) { return ((span + elems - 1) / elems + 31) / 32 * 32; }
inline int ctas_sm(int threads, int most) { return most / threads > 0 ? most / threads : 1; }

constexpr int kLateRows = 16, kLatePart = 8;   // late slots from so many rows a slot on; the part of all rows that they take
inline void spread(RowPlan& p, int64_t rows, int groups, int per_sm, bool may_late) {
    int64_t lines = (int64_t)kAddNormSMs * per_sm * p.slots_per_cta / groups / 8 * 8;
    if (lines < 8) lines = 8;
    if (lines > rows) lines = rows;
    p.slots = (int)lines * groups;
    // SMs are not equally fast at memory (a fixed share of 3 operands read and 2 written each took 135 us where CTAs that
    // start as others end took 122).  So the last rows may be left to as many slots again, which start on whichever SMs are done.
    const bool late = may_late && rows >= kLateRows * lines;
    p.late_slots = late ? p.slots : 0;
    p.early_rows = (int)(late ? rows - rows / kLatePart : rows);
    p.grid = (p.slots + p.late_slots + p.slots_per_cta - 1) / p.slots_per_cta;
}

inline int set_slots(BlockNormBwdArgs& a, const RowPlan& p) {   // and how many rows of shares there will be
    a.slots = p.slots;
    a.late_slots = p.late_slots;
    a.early_rows = p.early_rows;
    a.slots_per_cta = p.slots_per_cta;
    return (p.slots + p.late_slots) / a.groups;
}

// Rows of up to 256 columns take 8, 16 or 32 lanes of a warp, others a CTA (131072 x 256 with a residual 122 us, by CTAs of a warp
// 129; without 64, 71): 8 elements a thread up to 512 columns, or up to 1280 of fp32, then 16.  33.5 M elements with gate and fp32
// residual, 8 and 16 elements a thread: bf16 768 columns 145 and 121 us, 1024 140 and 132, 1280 137 and 124 (512 by single warps of 16:
// 198; by 8 133); fp32 768 columns 164 and 186, 1024 176 and 166, 1280 168 and 182, 2048 198 and 169.  Rows of no whole vectors: 765
// columns 188 and 154, without a residual 1023 columns 106 and 87, from 8 bits 1261 columns 148 and 138; but with a residual 1023
// columns 161 and 172, 1261 140 and 147 (their last warp's threads are idle), so 8 for those beyond 1024.
constexpr int kNarrowSpan = 512, kNarrowSpanLong = 1280;
inline RowPlan vector_plan(int span, int narrow) {
    RowPlan p = {};
    p.elems = span <= narrow ? kNarrowElems : kWideElems;
    p.lanes = span <= 64 ? 8 : span <= 128 ? 16 : span <= 256 ? 32 : 0;
    p.threads = p.lanes ? 128 : row_threads(span, p.elems);
    p.slots_per_cta = p.lanes ? 128 / p.lanes : 1;
    return p;
}
inline RowPlan loose_plan(int64_t rows, int size, int groups) {
    RowPlan p = {};
    p.elems = size <= 512 * kNarrowElems ? kNarrowElems : kWideElems;
    p.threads = row_threads(size, p.elems);
    p.slots_per_cta = p.threads == 32 ? 4 : 1;
    spread(p, rows, groups, ctas_sm(p.threads * p.slots_per_cta, loose_threads_sm(p.elems)), false);
    if (p.slots < p.slots_per_cta) p.slots_per_cta = p.slots;   // no late ones then
    p.threads *= p.slots_per_cta;
    return p;
}

template <typename T, typename R, int E, int LANES, bool SHIFTED, bool GATE, bool RES, bool XP, bool HP>
cudaError_t launch_ring(BlockNormBwdArgs& a, RowPlan p, int* lines, cudaStream_t st) {
    typedef Record<T, R, E, GATE, RES, XP, HP> Rec;
    auto kern = ssd_block_norm_bwd_kernel<T, R, E, LANES, SHIFTED, GATE, RES, XP, HP>;
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
    const int stage = p.threads * Rec::bytes, weights = p.threads * Rec::weights;
    int per_sm = ctas_sm(p.threads, threads_sm(E, RES));
    for (;; --per_sm) {
        const int room = (kSmemSM / per_sm < kSmemCta + 1024 ? kSmemSM / per_sm : kSmemCta + 1024) - 1024 - kSmemOwn;
        a.stages = (room - weights) / stage;
        if (a.stages >= (RES ? 1 : 2) || per_sm == 1) break;
    }
    if (a.stages < 1) return cudaErrorNotSupported;
    if (a.stages > (RES ? 1 : kMaxStages)) a.stages = RES ? 1 : kMaxStages;
    // Late slots where HBM is the bound and the shares are those of one weight: bf16 gate and norm 16384 x 5120 153 us without,
    // 140 with; 8192 x 80 groups of 64 81, 69; 16384 x 2048 63, 60.  From codes 124, 135; fp32 2048 columns 108, 112; one CTA an SM
    // (8192 columns) 59, 68; with a residual 16384 x 2560 166, 170.
    spread(p, a.rows, a.groups, per_sm, !RES && !XP && sizeof(T) == 2 && per_sm > 1);
    *lines = set_slots(a, p);
    if (*lines > a.share_lines) return cudaErrorInvalidValue;
    return launch_kernel(kern, (unsigned)p.grid, (unsigned)p.threads, (size_t)weights + (size_t)a.stages * stage, st, true, a);
}

template <typename T, typename R, bool SHIFTED, bool GATE, bool RES, bool XP, bool HP>
cudaError_t launch_vectors(BlockNormBwdArgs& a, int* lines, cudaStream_t st) {
    const int span = SHIFTED ? vector_span(a.size) : a.size;
    const RowPlan p = vector_plan(span, sizeof(T) == 4 || (SHIFTED && RES && !XP && span > 1024) ? kNarrowSpanLong : kNarrowSpan);
    if (p.lanes == 8) return launch_ring<T, R, kNarrowElems, 8, SHIFTED, GATE, RES, XP, HP>(a, p, lines, st);
    if (p.lanes == 16) return launch_ring<T, R, kNarrowElems, 16, SHIFTED, GATE, RES, XP, HP>(a, p, lines, st);
    if (p.lanes == 32) return launch_ring<T, R, kNarrowElems, 32, SHIFTED, GATE, RES, XP, HP>(a, p, lines, st);
    return p.elems == kNarrowElems ? launch_ring<T, R, kNarrowElems, 0, SHIFTED, GATE, RES, XP, HP>(a, p, lines, st)
                                   : launch_ring<T, R, kWideElems, 0, SHIFTED, GATE, RES, XP, HP>(a, p, lines, st);
}

// The main launch; *lines: rows of shares that it leaves.  Vectors where every array starts on 16 bytes (codes on a vector's), rows hold
// one at least, x and gate are both codes or neither is, and an SM's shared memory holds a row's records.
template <typename T, typename R, bool GATE, bool RES>
cudaError_t launch_block_norm_bwd_typed(BlockNormBwdArgs& a, int* lines, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    auto fits = [](const void* p, bool packed) { return ((uintptr_t)p & (packed ? V - 1 : 15)) == 0; };
    const bool shifted = a.size % V != 0;
    const int width = a.size * a.groups;
    const bool xp = a.x_scales, hp = RES && a.dout && a.h_scales;
    const bool vectors = a.size >= V && vector_span(a.size) <= 512 * kWideElems && fits(a.x, xp) && fits(a.h, hp) && fits(a.dout, false) &&
                         fits(a.dres, false) && fits(a.dres_out, false) && fits(a.dx, false) && fits(a.out, false) &&
                         (shifted || (fits(a.weight, false) && fits(a.next_weight, false))) &&
                         (!GATE || (xp == (a.gate_scales != nullptr) && fits(a.gate, xp) && fits(a.dgate, false) &&
                                    (shifted ? a.gate_stride == width && a.dgate_stride == width
                                             : a.gate_stride % V == 0 && a.dgate_stride % V == 0)));
    cudaError_t e = cudaErrorNotSupported;
    if (vectors && hp) {
        if constexpr (RES)
            e = xp ? (shifted ? launch_vectors<T, R, true, GATE, RES, true, true>(a, lines, st)
                              : launch_vectors<T, R, false, GATE, RES, true, true>(a, lines, st))
                   : (shifted ? launch_vectors<T, R, true, GATE, RES, false, true>(a, lines, st)
                              : launch_vectors<T, R, false, GATE, RES, false, true>(a, lines, st));
    } else if (vectors) {
        e = xp ? (shifted ? launch_vectors<T, R, true, GATE, RES, true, false>(a, lines, st)
                          : launch_vectors<T, R, false, GATE, RES, true, false>(a, lines, st))
               : (shifted ? launch_vectors<T, R, true, GATE, RES, false, false>(a, lines, st)
                          : launch_vectors<T, R, false, GATE, RES, false, false>(a, lines, st));
    }
    if (e != cudaErrorNotSupported) return e;   // not even one row's records fit an SM: the widest fp32 rows
    const RowPlan p = loose_plan(a.rows, a.size, a.groups);
    *lines = set_slots(a, p);
    if (*lines > a.share_lines) return cudaErrorInvalidValue;
    return launch_kernel(p.elems == kNarrowElems ? ssd_block_norm_bwd_loose<T, R, kNarrowElems, GATE, RES>
                                                 : ssd_block_norm_bwd_loose<T, R, kWideElems, GATE, RES>,
                         (unsigned)p.grid, (unsigned)p.threads, 0, st, true, a);
}

// One per file: the gate and norm after the scan; the norm after a block by types, without and with a gate.
cudaError_t launch_gate_norm_bwd_typed(BlockNormBwdArgs& a, int* lines, cudaStream_t st);
cudaError_t launch_block_norm_bwd_f32(BlockNormBwdArgs& a, int* lines, cudaStream_t st);
cudaError_t launch_block_norm_bwd_bf16_f32(BlockNormBwdArgs& a, int* lines, cudaStream_t st);
cudaError_t launch_block_norm_bwd_bf16(BlockNormBwdArgs& a, int* lines, cudaStream_t st);

}  // namespace ssd
