// flat_plan.cuh -- where a position of a batch's flat work order lies.
//
// The work of a call is one flat range of equal units, sequence after sequence
// (count(b) units for sequence b), cut into contiguous pieces of equal size.
// Every CTA finds its piece's first sequence itself from the lengths, so no
// plan kernel runs first.
#pragma once

#include "common.cuh"

namespace nvfp4kv {

__device__ __forceinline__ int clamp_rows(int32_t n, int64_t cap) { return n < 0 ? 0 : (int64_t)n > cap ? (int)cap : n; }

template <int T>
struct FlatScratch {
    int64_t prefix[T + 1];
    int64_t warp[T / 32];
};

// All T threads of the CTA call it.  count(b): units of sequence b.  want(total):
// this thread's position, given the number of units; on return b and first are
// its sequence and that sequence's first unit (b = B if the position is >= total
// or negative).  Returns the number of units.
template <int T, class Count, class Want>
__device__ __forceinline__ int64_t flat_locate(FlatScratch<T> &s, int B, Count count, Want want, int &b,
                                               int64_t &first) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // exclusive prefix of sequences c0 .. c0 + T - 1 (from `base`) into s.prefix; returns the end
    auto scan = [&](int c0, int64_t base) {
        int64_t v = c0 + tid < B ? (int64_t)count(c0 + tid) : 0;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, v, x);
            if (lane >= x) v += y;
        }
        if (lane == 31) s.warp[warp] = v;
        __syncthreads();
        int64_t before = base;
        for (int w = 0; w < warp; w++) before += s.warp[w];
        s.prefix[tid + 1] = before + v;
        if (tid == 0) s.prefix[0] = base;
        __syncthreads();
        return s.prefix[T];
    };
    b = B;
    first = 0;
    int64_t total = 0;
    for (int c0 = 0; c0 < B; c0 += T) {
        total = scan(c0, total);
        if (B > T) __syncthreads();   // the next scan overwrites what is read above
    }
    const int64_t u = want(total);
    int64_t base = 0;
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

// Piece i of `pieces` of a range of `total` units: [begin, end).
__device__ __forceinline__ int64_t flat_begin(int64_t i, int64_t total, int64_t pieces) { return i * total / pieces; }

// The piece that holds unit u (0 <= u < total).
__device__ __forceinline__ int64_t flat_piece(int64_t u, int64_t total, int64_t pieces) {
    return ((u + 1) * pieces - 1) / total;
}

}  // namespace nvfp4kv
