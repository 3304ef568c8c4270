// flat_plan.cuh -- where a position of a batch's flat work order lies.
//
// The work of a call is one flat range of equal units, sequence after sequence
// (count(b) units for sequence b; the host refuses 2^31 of them), cut into
// contiguous pieces whose sizes differ by at most one.  Every CTA finds its
// piece's first sequence itself from the lengths, so no plan kernel runs first.
#pragma once

#include "common.cuh"

namespace nvfp4kv {

__device__ __forceinline__ int clamp_rows(int32_t n, int64_t cap) { return n < 0 ? 0 : (int64_t)n > cap ? (int)cap : n; }

// `total` units in `pieces` pieces, the first total % pieces of them one unit larger.
struct FlatCut {
    unsigned q, r;
    __device__ __forceinline__ FlatCut(unsigned total, unsigned pieces) : q(total / pieces), r(total % pieces) {}
    __device__ __forceinline__ unsigned begin(unsigned i) const { return i * q + min(i, r); }
    __device__ __forceinline__ unsigned piece(unsigned u) const {   // that holds unit u < total
        const unsigned large = r * (q + 1);
        return u < large ? u / (q + 1) : r + (u - large) / q;
    }
};

template <int T>
struct FlatScratch {
    unsigned prefix[T + 1];
    unsigned warp[T / 32];
};

constexpr int kFlatWarp = 128;        // sequences that a warp scans by itself
constexpr unsigned kFlatNone = ~0u;   // no position

// All T threads of the CTA call it.  count(b): units of sequence b.  want(total): the
// warp's position, given the number of units; on return b and first are its sequence and
// that sequence's first unit (b = B if the position is none of the units').  Returns the
// number of units.  Up to kFlatWarp sequences each warp scans the lengths itself, without
// a barrier (with them, and 64-bit sums, locating took 1.9 us of a call, now 0.8).
template <int T, class Count, class Want>
__device__ __forceinline__ unsigned flat_locate(FlatScratch<T> &s, int B, Count count, Want want, int &b, unsigned &first) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto scan_warp = [&](unsigned v) {   // inclusive
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, v, x);
            if (lane >= x) v += y;
        }
        return v;
    };
    b = B;
    first = 0;
    if (B <= kFlatWarp) {
        constexpr int K = kFlatWarp / 32;   // lane: sequences K lane .. K lane + K - 1
        unsigned c[K], sum = 0;
#pragma unroll
        for (int k = 0; k < K; k++) c[k] = K * lane + k < B ? (unsigned)count(K * lane + k) : 0u;
#pragma unroll
        for (int k = 0; k < K; k++) sum += c[k];
        const unsigned end = scan_warp(sum), total = __shfl_sync(0xffffffffu, end, 31);
        const unsigned u = want(total);
        if (u >= total) return total;
        unsigned at = end - sum;
        const int holder = 31 - __clz(__ballot_sync(0xffffffffu, at <= u));   // the last lane that starts at or below u
        int own = K * lane;
        bool on = true;
#pragma unroll
        for (int k = 0; k < K - 1; k++) {
            on = on && at + c[k] <= u;
            if (on) {
                at += c[k];
                own++;
            }
        }
        b = __shfl_sync(0xffffffffu, own, holder);
        first = __shfl_sync(0xffffffffu, at, holder);
        return total;
    }
    // exclusive prefix of sequences c0 .. c0 + T - 1 (from `base`) into s.prefix; returns the end
    auto scan = [&](int c0, unsigned base) {
        const unsigned v = scan_warp(c0 + tid < B ? (unsigned)count(c0 + tid) : 0u);
        if (lane == 31) s.warp[warp] = v;
        __syncthreads();
        unsigned before = base;
        for (int w = 0; w < warp; w++) before += s.warp[w];
        s.prefix[tid + 1] = before + v;
        if (tid == 0) s.prefix[0] = base;
        __syncthreads();
        return s.prefix[T];
    };
    unsigned total = 0;
    for (int c0 = 0; c0 < B; c0 += T) {
        total = scan(c0, total);
        if (B > T) __syncthreads();   // the next scan overwrites what is read above
    }
    const unsigned u = want(total);
    unsigned base = 0;
    for (int c0 = 0; c0 < B; c0 += T) {
        if (B > T) base = scan(c0, base);
        if (u >= s.prefix[0] && u < s.prefix[T]) {
            int lo = 0, hi = T - 1;   // the last entry with prefix <= u: its sequence holds the unit
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s.prefix[mid] <= u) lo = mid;
                else hi = mid - 1;
            }
            b = c0 + lo;
            first = s.prefix[lo];
        }
        __syncthreads();
    }
    return total;
}

}  // namespace nvfp4kv
