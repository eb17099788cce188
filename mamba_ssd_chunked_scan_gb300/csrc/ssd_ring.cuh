// Rows that come through shared memory ahead of their use (sm_103a): each thread copies its own vectors of the rows to come into
// records of its warp (cp.async) and reads them there as often as it needs.  No barrier and no register holds them.
//
// Rows of n elements, n not a multiple of a vector's V (SHIFTED): vectors lie on V-element boundaries of the whole array, and a row
// starts `shift` elements into its first one.  That one holds the row before's last elements too, which are read with it
// (and cleared) and never written; what the last one holds of the next row is not read.  The rows that a thread walks are
// a multiple of 8 apart, so that their shift is one number and the thread's columns stay its own.
#pragma once
#include "ssd_rows.cuh"

namespace ssd {

constexpr int kWideElems = 16, kNarrowElems = 8;   // elements of a row per thread
constexpr int kSmemSM = 228 * 1024, kSmemCta = 227 * 1024;
constexpr int kSmemOwn = 2048;                     // a CTA's static shared memory and what the system takes

// Columns that the vectors of a row span: rows of other than whole vectors may reach into one more.
inline int vector_span(int size) { return size % 8 == 0 ? size : size + 7; }

// Copies of 16, 8 or 4 bytes, of which the first `n` are read and the others 0.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int n) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most the newest `n` groups of copies are under way.
__device__ __forceinline__ void copies_wait(int n) {
    if (n == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <bool, typename A, typename B> struct Pick { typedef A type; };
template <typename A, typename B> struct Pick<false, A, B> { typedef B type; };

// Where the 16-byte half `k` of a lane's vector c of type K lies, or all of it where K is shorter, from an operand's first piece on.
// Vectors of 32 bytes (fp32 beside bf16) are copied by pairs of lanes, 32 adjacent bytes at a time: a lane that took its own two
// halves would ask for each 32-byte sector twice (588 MB of operands, half of them so, took 148 us).  The order of their places
// keeps both the copies and the reads off each other's banks.
template <typename K, int V>
__device__ __forceinline__ int piece(int c, int k, int lane) {
    constexpr int kBytes = (int)sizeof(K) * V;
    if constexpr (kBytes == 32) return (c * 2 + (lane & 1)) * 512 + (((lane & 30) | k) ^ (lane & 1)) * 16;
    else return (c * 32 + lane) * kBytes;
}

// One vector (number c of the lane's) of an operand, whose pieces start at `at`.
template <typename K, int V>
__device__ __forceinline__ Raw<K, V> piece_vector(const unsigned char* at, int c, int lane) {
    Raw<K, V> q;
    if constexpr (sizeof(K) * V == 32) {
        q.w.lo = *reinterpret_cast<const uint4*>(at + piece<K, V>(c, 0, lane));
        q.w.hi = *reinterpret_cast<const uint4*>(at + piece<K, V>(c, 1, lane));
    } else {
        q.w = *reinterpret_cast<const typename Raw<K, V>::W*>(at + piece<K, V>(c, 0, lane));
    }
    return q;
}
// Ask for the elements of vector c (from column e, `off` bytes from p) that lie before the row's end, n, into its pieces, and zeros for
// the others: vectors of one lane each for itself, 32-byte ones with the neighbouring lane.  A vector past the end is left alone.
template <typename K, int V, bool SHIFTED>
__device__ __forceinline__ void ask(uint32_t to, int c, int lane, const unsigned char* p, uint32_t off, int e, int n) {
    constexpr int kBytes = (int)sizeof(K) * V;
    if constexpr (kBytes == 32) {
        const int k = lane & 1;
        const unsigned char* pair = p + (off - 32 * k);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int eo = e + (h - k) * V;   // the vector of the pair's lane h
            if (eo >= n) continue;
            const int bytes = SHIFTED ? max(0, min(16, (n - eo - k * V / 2) * (int)sizeof(K))) : 16;
            copy_async<16>(to + piece<K, V>(c, k, (lane & 30) | h), pair + (SHIFTED && bytes == 0 ? 0 : 32 * h + 16 * k), bytes);
        }
    } else {
        if (e >= n) return;
        const int bytes = SHIFTED ? min(kBytes, (n - e) * (int)sizeof(K)) : kBytes;
        copy_async<kBytes>(to + piece<K, V>(c, 0, lane), p + off, bytes);
    }
}

// 0 in the first `cut` elements of a vector, which belong to the row before.
template <typename K, int V>
__device__ __forceinline__ void clear_head(unsigned char* at, int c, int lane, int cut) {
    constexpr int kWords = (int)sizeof(K) * V / 4, kEach = kWords > 4 ? 4 : kWords;   // words of the vector, of a piece
    const int bytes = cut * (int)sizeof(K);
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
        uint32_t* w = reinterpret_cast<uint32_t*>(at + piece<K, V>(c, j / kEach, lane)) + j % kEach;
        const int b = bytes - 4 * j;   // bytes of the word to clear
        if (b >= 4) *w = 0;
        else if (b > 0) *w &= 0xffffffffu << (8 * b);
    }
}

// Store the elements of a vector (from column e, `off` bytes from `row`) that lie in a row's columns [0, n); 32-byte vectors with the
// neighbouring lane, as they are copied (all lanes of `mask` call).
template <typename K, int V, bool SHIFTED>
__device__ __forceinline__ void put(unsigned char* row, uint32_t off, int e, int n, uint32_t mask, const Two (&v)[V / 2]) {
    Raw<K, V> q;
    from_pairs(v, q);
    if constexpr ((int)sizeof(K) * V == 32) {
        const int k = threadIdx.x & 1;
        uint4 keep = k ? q.w.hi : q.w.lo, give = k ? q.w.lo : q.w.hi;
        give.x = __shfl_xor_sync(mask, give.x, 1);
        give.y = __shfl_xor_sync(mask, give.y, 1);
        give.z = __shfl_xor_sync(mask, give.z, 1);
        give.w = __shfl_xor_sync(mask, give.w, 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int eo = e + (h - k) * V + k * (V / 2);   // the first column of the half
            Raw<K, V / 2> r;
            r.w = h == k ? keep : give;
            K* p = reinterpret_cast<K*>(row + (off - 32 * k + 32 * h + 16 * k));
            if constexpr (SHIFTED) {
                if (eo >= 0 && eo + V / 2 <= n) r.store(p);
                else r.store_within(p - eo, eo, n);
            } else {
                if (eo < n) r.store(p);
            }
        }
    } else {
        K* p = reinterpret_cast<K*>(row + off);
        if constexpr (SHIFTED) {
            if (e >= 0 && e + V <= n) q.store(p);
            else q.store_within(p - e, e, n);
        } else {
            if (e < n) q.store(p);
        }
    }
}

}  // namespace ssd
