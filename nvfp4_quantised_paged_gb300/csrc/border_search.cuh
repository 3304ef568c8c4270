// border_search.cuh -- the search for the border between kept and dropped keys (evict.cu).
//
// Host code too (plain C++ where __host__ and __device__ mean nothing): how keys are counted
// is the caller's.
#pragma once

#include <stdint.h>

namespace nvfp4kv {

// The largest border with at least `want` >= 1 keys not below it, two bits a step down to bit
// `last`; it starts with the bits of `border` above bit `top`.  count(border, bit, step, c)
// sets c[x] to the keys not below border | x << bit, x = 1 .. 3.  exact: the search ended at a
// border with just `want` keys not below it.
template <class Count>
__host__ __device__ __forceinline__ uint32_t search_pairs(uint32_t border, int top, int last, uint32_t want, bool &exact,
                                                          Count count) {
    exact = false;
    int step = 0;
    for (int bit = top & ~1; bit >= last; bit -= 2, step++) {
        uint32_t c[4];
        count(border, bit, step, c);
        const uint32_t x = c[3] >= want ? 3u : c[2] >= want ? 2u : c[1] >= want ? 1u : 0u;
        border |= x << bit;
        if ((x == 3 ? c[3] : x == 2 ? c[2] : x == 1 ? c[1] : 0u) == want) {   // (want >= 1)
            exact = true;
            break;
        }
    }
    return border;
}

// The same over a list of keys lo <= key < hi that is searched alone, `want` at most their
// number.  The first trials, lo with its low bits cleared, may lie below lo: where all of the
// list is wanted one of them ends the search, and keys outside the list lie between it and lo.
// No listed key does, so lo is the border then.
template <class Count>
__host__ __device__ __forceinline__ uint32_t search_listed(uint32_t lo, uint32_t hi, uint32_t want, bool &exact, Count count) {
    int top = -1;                               // the highest bit in which listed keys differ
    for (uint32_t diff = lo ^ (hi - 1u); diff; diff >>= 1) top++;
    const uint32_t border = top >= 0 ? lo & ~((4u << (top & ~1)) - 1u) : lo;   // (4 << 30: 0, all bits are open)
    const uint32_t found = search_pairs(border, top, 0, want, exact, count);
    return found < lo ? lo : found;
}

}  // namespace nvfp4kv
