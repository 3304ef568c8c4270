// evict.cu -- the tokens of largest score of every sequence and kv head, moved into new pages.
//
// Two kernels:
//   select   finds the smallest kept key of each (sequence, kv head) with n > keep rows
//            over the scores' order-preserving 32-bit keys.  Rows that must stay (the
//            first `sink`, the last `recent`) have the largest key; ties at the border
//            go to the lowest index; the kept indices are written in order.  Up to 32,768
//            rows one CTA holds the keys in registers (select_one_kernel).  Longer
//            segments take a cluster of up to eight CTAs and a radix select of 8 bits a
//            round: each CTA counts its part of the rows in shared memory, the cluster
//            adds the 256 counts up through distributed shared memory and every CTA picks
//            the same digit; then each warp counts and compacts a contiguous part of the
//            rows, its offset coming from one scan over the CTA's warps and one over the
//            cluster.  Keys stay in shared memory between the rounds as far as they fit;
//            where they do not, a sample's borders take the place of the rounds here too.
//            (16 x 8 segments of up to 32,768 rows: 23 us with one CTA each, 66 us with
//            clusters of four.)  Which it is goes by the rows that the table and the score
//            rows have room for: the lengths are on the device.
//   move     one warp per 16-row group of the new pages gathers its rows and writes the
//            group's contiguous bytes: 36 us for 524,288 rows, which read 288 bytes of
//            32-byte sectors each for their 144 and write 144: 6.3 TB/s.
// Nothing is atomic in global memory, so the result does not depend on timing.
#include <cooperative_groups.h>

#include <mutex>

#include "border_search.cuh"
#include "common.cuh"
#include "flat_plan.cuh"
#include "kernels.h"

namespace nvfp4kv {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kKeyCache = 16384;            // keys of a CTA's part kept in shared memory (64 KB)
constexpr int kMaxCluster = 8;

// CTAs that a launch of clusters aims at, two per SM of a 152-SM GPU.  (16 x 8 segments of
// 40,000 rows: 107 us with 304, 171 us with 152, 118 us with 608; one segment: 24 us as a
// cluster of eight, 164 us alone.)
constexpr int kTargetCtasSel = 304;

struct SelectArgs {
    const float *scores;
    int64_t score_stride;
    int B, Hkv;
    const int32_t *seq_lens;
    int64_t cap;                // rows a sequence may have: min(table, score_stride)
    int keep, recent, sink;
    int32_t *new_lens, *kept;
    float *new_scores;
    int64_t new_score_stride;
    unsigned *err;
};

// Keys order as the scores do (-0 below +0 would split equal scores: both give
// the key of 0); a NaN gets 1, below -inf (0: no row).
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 1u;
    const uint32_t u = __float_as_uint(x + 0.0f);   // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// What both selections write around the kept rows of a segment: its new length, -1
// and score 0 behind it, and, where every row stays, all of it (true is returned).
__device__ __forceinline__ bool select_edges(const SelectArgs &a, int seg, int n, int32_t len, int first, int step,
                                             const float *src, int32_t *kept, float *dst) {
    const int new_n = min(n, a.keep);
    if (first == 0 && seg % a.Hkv == 0) {
        a.new_lens[seg / a.Hkv] = new_n;
        if (len < 0 || (int64_t)len > a.cap) flag_error(a.err, kErrSeqLen);
    }
    for (int i = new_n + first; i < a.keep; i += step) kept[i] = -1;
    const int64_t end = a.new_score_stride;
    int64_t i0 = new_n;                       // zeros: single ones up to a 16-byte boundary, then four at a time
    while (i0 < end && (reinterpret_cast<uintptr_t>(dst + i0) & 15)) {
        if (first == 0) dst[i0] = 0.f;
        i0++;
    }
    for (int64_t i = i0 + 4 * (int64_t)first; i < end; i += 4 * (int64_t)step) {
        if (i + 4 <= end) {
            *reinterpret_cast<float4 *>(dst + i) = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            for (int64_t x = i; x < end; x++) dst[x] = 0.f;
        }
    }
    if (n > a.keep) return false;
    for (int i = first; i < n; i += step) {
        kept[i] = i;
        dst[i] = src[i];
    }
    return true;
}

// One CTA a segment of up to kOneRows rows: every thread holds PER consecutive
// keys in registers, and the border key is found bit by bit, a count over the CTA
// each (counting digits in shared memory took 40 clocks a warp and 32 keys).  Most
// of the rows are left out of that search: 512 keys spread over the rows are a
// sample whose ranks, found by one warp, give two keys between which the border
// almost always lies; one count over all rows confirms it, and the few keys between
// them are searched alone.  (Where they do not, all keys are.)  The search ends as soon
// as a border splits off exactly the rows wanted.  A thread's kept rows are consecutive
// too: one scan places them all.
// 256 threads up to 8,192 rows (several CTAs an SM, cheaper sums), 1,024 beyond.
constexpr int kOnePer = 33;                  // odd: consecutive keys of 32 threads lie in 32 banks
constexpr int kOneSmall = 256, kOneLarge = 1024;
constexpr int kOneSmallRows = kOneSmall * (kOnePer - 1), kOneRows = kOneLarge * (kOnePer - 1);
constexpr int kListPer = 8;                  // keys a thread has of the list between the two borders
constexpr int kSample = 512, kSamplePer = kSample / 32;
constexpr int kSampleBits = 20;              // of a sample border that are found (sign, exponent, 11 of the fraction)

// Sum of c over the CTA's T threads; buf alternates between calls.
template <int T>
__device__ __forceinline__ uint32_t cta_sum(uint32_t c, uint32_t (&s_count)[2][32], int buf) {
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0) s_count[buf][threadIdx.x >> 5] = c;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < T / 32 ? s_count[buf][threadIdx.x & 31] : 0u);
}

// Exclusive sum of v over the CTA's threads before this one, and the total.
template <int T>
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t (&s_count)[2][32], uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl += y;
    }
    __syncthreads();                          // s_count is read
    if (lane == 31) s_count[0][warp] = incl;
    __syncthreads();
    uint32_t w = lane < T / 32 ? s_count[0][lane] : 0u;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, x);
        if (lane >= x) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    __syncthreads();                          // s_count may be written again
    return (warp ? before : 0u) + incl - v;
}

// The largest border with at least `want` >= 1 of the CTA's keys (K a thread) not below it;
// exact: there are just `want`.  The border has the bits of `border` above bit `top`.
template <int T, int K>
__device__ __forceinline__ uint32_t find_border(const uint32_t (&k)[K], uint32_t want, uint32_t border, int top,
                                                uint32_t (&s_count)[2][32], bool &exact) {
    exact = false;
    for (int bit = top; bit >= 0; bit--) {
        const uint32_t trial = border | (1u << bit);
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < K; i++) c += k[i] >= trial;
        c = cta_sum<T>(c, s_count, bit & 1);
        if (c >= want) border = trial;
        if (c == want) {
            exact = true;
            break;
        }
    }
    return border;
}

// Counts of a step of search_pairs over the CTA, for few keys a thread (`used` of them, the others are 0): the warp's counts
// of the three trials, up to 32 K each, share a word (one bit a step took 4.0 us of the 32,768-row segments' 25).
template <int T, int K>
__device__ __forceinline__ void count_pairs(const uint32_t (&k)[K], int used, uint32_t border, int bit, int buf,
                                            uint32_t (&s_count)[2][32], uint32_t (&n)[4]) {
    static_assert(32 * K < 1024, "a warp's count must fit ten bits");
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < K; i++) {
        if (i >= used) break;
#pragma unroll
        for (uint32_t x = 1; x < 4; x++) c += k[i] >= (border | (x << bit)) ? 1u << (10 * (x - 1)) : 0u;
    }
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0) s_count[buf][threadIdx.x >> 5] = c;
    __syncthreads();
    c = (threadIdx.x & 31) < T / 32 ? s_count[buf][threadIdx.x & 31] : 0u;
    n[1] = __reduce_add_sync(0xffffffffu, c & 1023u);
    n[2] = __reduce_add_sync(0xffffffffu, (c >> 10) & 1023u);
    n[3] = __reduce_add_sync(0xffffffffu, c >> 20);
}

template <int T, int PER>
__device__ __forceinline__ void select_rows(const SelectArgs &a, int n, int per, int32_t *kept, uint32_t *s_keys,
                                            uint32_t (&s_count)[2][32]) {
    const int t0 = (int)threadIdx.x * per, last = n - a.recent;
    const uint32_t keep = (uint32_t)a.keep;
    auto key_at = [&](int t) { return t < a.sink || t >= last ? 0xffffffffu : score_key(__uint_as_float(s_keys[t])); };
    if (PER > 5 && threadIdx.x < 64) {   // (while the other warps lay out their keys)
        // sample ranks r -+ d around the border's expected one: warp 0 finds the upper border, warp 1 the lower
        const int lane = (int)threadIdx.x & 31, low = (int)threadIdx.x >> 5;
        uint32_t x[kSamplePer];
#pragma unroll
        for (int i = 0; i < kSamplePer; i++) x[i] = key_at((int)((int64_t)n * (i * 32 + lane) / kSample));
        const int r = (int)((int64_t)keep * kSample / n), d = 4 + (int)(3.0f * sqrtf((float)r));
        const uint32_t want = (uint32_t)(low ? min(r + d, kSample) : max(r - d, 0));
        uint32_t found_at = 0;
        for (int bit = 31; bit > 31 - kSampleBits; bit--) {
            const uint32_t trial = found_at | (1u << bit);
            uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kSamplePer; i++) c[i & 3] += x[i] >= trial;
            if (__reduce_add_sync(0xffffffffu, (c[0] + c[1]) + (c[2] + c[3])) >= want) found_at = trial;
        }
        // (the upper one no lower than the sample's border; no carry: the low bits are 0)
        if (lane == 0) s_count[1][low] = low ? found_at : found_at + ((1u << (32 - kSampleBits)) - 1u);
    }
    uint32_t k[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) k[i] = i < per && t0 + i < n ? key_at(t0 + i) : 0u;   // (0: below every border)
    uint32_t border = 0;
    bool exact = false, found = false;
    if (PER > 5) {
        __syncthreads();
        const uint32_t hi = s_count[1][0], lo = s_count[1][1];
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < PER; i++) c += (k[i] >= hi ? 1u : 0u) + (k[i] >= lo ? 0x10000u : 0u);
        const uint32_t own = (c >> 16) - (c & 0xffffu);   // lo <= key < hi
        c = cta_sum<T>(c, s_count, 0);           // (both at most kOneRows)
        const uint32_t c_hi = c & 0xffffu, c_lo = c >> 16;
        if (lo > 0 && c_hi < keep && keep <= c_lo && c_lo - c_hi <= T * kListPer) {
            uint32_t total;
            uint32_t at = cta_scan<T>(own, s_count, total);
#pragma unroll
            for (int i = 0; i < PER; i++)
                if (k[i] - lo < hi - lo) s_keys[at++] = k[i];   // (every thread has read its keys)
            __syncthreads();
            uint32_t x[kListPer];
#pragma unroll
            for (int i = 0; i < kListPer; i++)
                x[i] = threadIdx.x + i * T < total ? s_keys[threadIdx.x + i * T] : 0u;
            const int used = ((int)total + T - 1) / T;
            border = search_listed(lo, hi, keep - c_hi, exact, [&](uint32_t at_least, int bit, int step, uint32_t (&c)[4]) {
                count_pairs<T>(x, used, at_least, bit, step & 1, s_count, c);
            });
            found = true;
        }
    }
    if (!found) {
        __syncthreads();
        border = find_border<T>(k, keep, 0u, 31, s_count, exact);
    }
    // rows above the border stay, and of those equal to it the first keep - (rows above)
    const uint32_t from = exact ? border : border + 1u;   // (no overflow: a border of all ones is exact or never tried)
    uint64_t take = 0, even = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        if (k[i] >= from) take |= 1ull << i;
        if (k[i] == border) even |= 1ull << i;
    }
    if (exact) even = 0;
    const uint32_t gt = (uint32_t)__popcll((long long)take), eq = (uint32_t)__popcll((long long)even);
    uint32_t total;                           // (both counts fit 16 bits: at most kOneRows)
    const uint32_t before = cta_scan<T>(gt | (eq << 16), s_count, total);
    total &= 0xffffu;
    const uint32_t need = keep - total;       // 0 if the border was exact
    const uint32_t eqs = before >> 16;
    uint32_t at = (before & 0xffffu) + min(eqs, need);
    uint32_t ties = eqs < need ? need - eqs : 0u;         // of this thread's ties, the first so many stay
    while (even && ties > 0) {
        take |= even & (0ull - even);
        even &= even - 1;
        ties--;
    }
    while (take && at < keep) {               // (one step a kept row of the fullest thread, not one a row)
        kept[at++] = t0 + __ffsll((long long)take) - 1;
        take &= take - 1;
    }
}

// dst[i] = src[kept[i]] for this CTA's rows i in [c0, c1), written by its threads before (loads beside the
// compaction would stop each of its steps).
template <int T>
__device__ __forceinline__ void gather_scores(uint32_t c0, uint32_t c1, const float *src, const int32_t *kept, float *dst) {
    __syncthreads();
    for (uint32_t i = c0 + threadIdx.x; i < c1; i += T * 4) {
        int t[4];
#pragma unroll
        for (int e = 0; e < 4; e++) t[e] = i + e * T < c1 ? kept[i + e * T] : 0;
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (i + e * T < c1) dst[i + e * T] = __ldg(src + t[e]);
    }
}

template <int T>
__global__ void __launch_bounds__(T) select_one_kernel(SelectArgs a) {
    extern __shared__ __align__(16) uint32_t s_keys[];   // the scores' bits; later the keys between two borders
    __shared__ uint32_t s_count[2][32];
    pdl_wait();                                     // scores and lengths may be earlier work's
    pdl_launch_dependents();                        // (the move waits for this grid to complete)
    const int seg = (int)blockIdx.x, tid = threadIdx.x;
    const int32_t len = a.seq_lens[seg / a.Hkv];
    const int n = clamp_rows(len, a.cap);
    const float *src = a.scores + (int64_t)seg * a.score_stride;
    int32_t *kept = a.kept + (int64_t)seg * a.keep;
    float *dst = a.new_scores + (int64_t)seg * a.new_score_stride;
    // the scores by asynchronous copies, all in flight at once, while what lies around the kept rows is written
    if (n > a.keep && (a.score_stride & 3) == 0 && (reinterpret_cast<uintptr_t>(a.scores) & 15) == 0) {
        for (int t = 4 * tid; t < n; t += 4 * T)   // (a last one may pass n, not the row)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(s_keys + t)), "l"(src + t) : "memory");
    } else if (n > a.keep) {
        for (int t = tid; t < n; t += T)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(s_keys + t)), "l"(src + t) : "memory");
    }
    if (select_edges(a, seg, n, len, tid, T, src, kept, dst)) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    const int per = ((n + T - 1) / T) | 1;
    if (per <= 5)
        select_rows<T, 5>(a, n, per, kept, s_keys, s_count);
    else if (per <= 17)
        select_rows<T, 17>(a, n, per, kept, s_keys, s_count);
    else
        select_rows<T, kOnePer>(a, n, per, kept, s_keys, s_count);
    gather_scores<T>(0, (uint32_t)a.keep, src, kept, dst);
}

// Counts of a step of search_pairs over the keys of a cluster's CTAs: theirs are added up in
// distributed shared memory, one cluster barrier a step.
template <int K>
__device__ __forceinline__ void count_pairs_cluster(cg::cluster_group &cluster, const uint32_t (&k)[K], uint32_t border,
                                                    int bit, int buf, uint32_t (&s_count)[2][32],
                                                    uint32_t (&s_step)[2][4], uint32_t (&n)[4]) {
    const int lane = threadIdx.x & 31, C = (int)cluster.num_blocks();
    count_pairs<kSelThreads>(k, K, border, bit, buf, s_count, n);
    if (threadIdx.x == 0) {
#pragma unroll
        for (int x = 1; x < 4; x++) s_step[buf][x] = n[x];
    }
    cluster.sync();                                 // (a buffer is written again only after the next step's)
    const uint32_t *o = cluster.map_shared_rank(&s_step[0][0], lane < C ? lane : 0) + 4 * buf;
#pragma unroll
    for (int x = 1; x < 4; x++) n[x] = __reduce_add_sync(0xffffffffu, lane < C ? o[x] : 0u);
}

constexpr int kSampleLong = 2 * kSelThreads;        // keys that place the borders of a cluster's rows
constexpr int kSampleLast = 12;                     // bits of those borders that are left open
constexpr int kListLong = kSelThreads * kListPer;   // keys between them that a CTA holds

// kSampled: for launches in which a CTA may have more than kKeyCache rows.  (The other instance
// needs less of an SM: 16 x 8 segments of 40,000 rows took 130 us with one for both, 108 so.)
template <bool kSampled>
__global__ void __launch_bounds__(kSelThreads) select_kernel(SelectArgs a) {
    extern __shared__ uint32_t s_keys[];            // [kKeyCache]
    __shared__ uint32_t s_hist[256];                // this CTA's counts of a round; read by the cluster
    __shared__ uint32_t s_sum[256];
    __shared__ uint32_t s_warp[kSelWarps][2];       // kept-for-sure and border keys of each warp's part
    __shared__ uint32_t s_cta[2];                   // their sums; read by the cluster
    __shared__ uint32_t s_digit[2];
    pdl_wait();
    pdl_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
    const int seg = (int)blockIdx.y;                // b * Hkv + h
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t len = a.seq_lens[seg / a.Hkv];
    const int n = clamp_rows(len, a.cap);
    const float *src = a.scores + (int64_t)seg * a.score_stride;
    int32_t *kept = a.kept + (int64_t)seg * a.keep;
    float *dst = a.new_scores + (int64_t)seg * a.new_score_stride;
    if (select_edges(a, seg, n, len, rank * kSelThreads + tid, C * kSelThreads, src, kept, dst))
        return;                                     // uniform over the cluster
    // this CTA's rows [r0, r1), this warp's [w0, w1)
    const int per = (n + C - 1) / C;
    const int r0 = min(n, rank * per), r1 = min(n, r0 + per);
    const int wper = ((r1 - r0 + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int w0 = min(r1, r0 + warp * wper), w1 = min(r1, w0 + wper);
    const int last = n - a.recent;
    auto make_key = [&](int t) { return t < a.sink || t >= last ? 0xffffffffu : score_key(__ldg(src + t)); };
    auto key_of = [&](int t) { return t - r0 < kKeyCache ? s_keys[t - r0] : make_key(t); };

    uint32_t prefix = 0;                            // digits of the border key found so far
    uint32_t need = (uint32_t)a.keep;               // rows still to take among the keys with that prefix
    // As in one CTA, a sample gives two keys between which the border almost always lies: one pass
    // counts the keys above and lists those between, which are searched alone.  Where a CTA's keys
    // all stay in shared memory, the rounds below are quicker (2 x 262,144 rows: 133 us by rounds, 83 so;
    // 32 x 65,536: 46 and 61).
    bool found = false;
    if (kSampled && per > kKeyCache) {              // (uniform over the cluster)
        __shared__ uint32_t s_list[kSampled ? kListLong : 1];     // keys between the sampled borders
        __shared__ uint32_t s_count[2][32], s_step[2][4];
        __shared__ uint32_t s_between, s_sums[2];   // this CTA's: keys between, (keys above, between); the last read by the cluster
        uint32_t x[2];
#pragma unroll
        for (int i = 0; i < 2; i++) x[i] = make_key((int)((int64_t)n * (tid + i * kSelThreads) / kSampleLong));
        const int r = (int)((int64_t)a.keep * kSampleLong / n), d = 4 + (int)(3.0f * sqrtf((float)r));
        auto count = [&](uint32_t border, int bit, int step, uint32_t (&c)[4]) {
            count_pairs<kSelThreads>(x, 2, border, bit, step & 1, s_count, c);
        };
        uint32_t hi = 0xffffffffu;
        bool exact;
        if (r > d)
            hi = search_pairs(0u, 31, kSampleLast, (uint32_t)(r - d), exact, count) | ((1u << kSampleLast) - 1u);
        __syncthreads();
        const uint32_t lo = search_pairs(0u, 31, kSampleLast, (uint32_t)min(r + d, kSampleLong), exact, count);
        if (tid == 0) s_between = 0;
        __syncthreads();
        uint32_t above = 0;
        for (int tw = w0; tw < w1; tw += 128) {
            uint32_t k[4];
#pragma unroll
            for (int e = 0; e < 4; e++) k[e] = tw + 32 * e + lane < w1 ? make_key(tw + 32 * e + lane) : 0u;   // (0: below lo)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int t = tw + 32 * e + lane;
                if (t < w1 && t - r0 < kKeyCache) s_keys[t - r0] = k[e];   // read back by this thread only
                above += k[e] >= hi;
                const bool in = k[e] - lo < hi - lo;
                const unsigned ins = __ballot_sync(0xffffffffu, in && lo > 0);
                if (ins) {
                    uint32_t at = 0;
                    if (lane == 0) at = atomicAdd(&s_between, (uint32_t)__popc(ins));   // (their order says nothing)
                    at = __shfl_sync(0xffffffffu, at, 0) + (uint32_t)__popc(ins & ((1u << lane) - 1u));
                    if (in && at < (uint32_t)kListLong) s_list[at] = k[e];
                }
            }
        }
        above = cta_sum<kSelThreads>(above, s_count, 0);   // (its barrier: s_between and s_list are complete)
        const uint32_t own = s_between;
        if (tid == 0) {
            s_sums[0] = above;
            s_sums[1] = own <= (uint32_t)kListLong ? own : 0x1000000u;      // too many: no CTA goes on
        }
        cluster.sync();
        const uint32_t *o = cluster.map_shared_rank(s_sums, lane < C ? lane : 0);
        above = __reduce_add_sync(0xffffffffu, lane < C ? o[0] : 0u);
        const uint32_t between = __reduce_add_sync(0xffffffffu, lane < C ? o[1] : 0u);
        if (lo > 0 && between < 0x1000000u && above < need && need <= above + between) {
            uint32_t k[kListPer];
#pragma unroll
            for (int i = 0; i < kListPer; i++) k[i] = tid + i * kSelThreads < (int)own ? s_list[tid + i * kSelThreads] : 0u;
            const uint32_t border =
                search_listed(lo, hi, need - above, exact, [&](uint32_t at_least, int bit, int step, uint32_t (&c)[4]) {
                    count_pairs_cluster(cluster, k, at_least, bit, step & 1, s_count, s_step, c);
                });
            if (exact) {                            // just `keep` keys are not below the border
                prefix = border - 1u;               // (border > 0: not every key is kept)
                need = 0;
            } else {                                // the border is a key, of which the first ones are taken
                uint32_t c = 0;
#pragma unroll
                for (int i = 0; i < kListPer; i++) c += k[i] > border;
                cluster.sync();                     // (s_sums is read)
                c = cta_sum<kSelThreads>(c, s_count, 0);
                if (tid == 0) s_sums[0] = c;
                cluster.sync();
                c = __reduce_add_sync(0xffffffffu, lane < C ? o[0] : 0u);
                prefix = border;
                need -= above + c;
            }
            found = true;
        }
        cluster.sync();                             // (s_sums and s_step are read)
    }
    for (int round = 0; round < 4 && !found; round++) {
        const int shift = 24 - 8 * round;
        if (tid < 256) s_hist[tid] = 0;
        __syncthreads();
        for (int tw = w0; tw < w1; tw += 32) {
            const int t = tw + lane;
            uint32_t k = 0;
            bool in = t < w1;
            if (in && round == 0) {
                k = make_key(t);
                if (t - r0 < kKeyCache) s_keys[t - r0] = k;   // read back by this thread only
            } else if (in) {
                k = key_of(t);
                in = (k >> (shift + 8)) == prefix;
            }
            // counts of equal digits are added by one lane (scores share exponents: plain atomics would queue)
            const uint32_t d = in ? (k >> shift) & 255u : 256u;
            const unsigned peers = __match_any_sync(0xffffffffu, d);
            if (in && lane == __ffs(peers) - 1) atomicAdd(&s_hist[d], (uint32_t)__popc(peers));
        }
        cluster.sync();
        if (tid < 256) {
            uint32_t sum = 0;
            for (int r = 0; r < C; r++) sum += cluster.map_shared_rank(s_hist, r)[tid];
            s_sum[tid] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            // the digit whose keys cross `need`, counted from the largest: lane i owns digits 255 - 8i .. 248 - 8i
            uint32_t own = 0;
#pragma unroll
            for (int x = 0; x < 8; x++) own += s_sum[255 - 8 * lane - x];
            uint32_t incl = own;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, x);
                if (lane >= x) incl += y;
            }
            uint32_t above = incl - own;
            if (above < need && need <= incl) {
                for (int x = 0; x < 8; x++) {
                    const uint32_t c = s_sum[255 - 8 * lane - x];
                    if (above + c >= need) {
                        s_digit[0] = 255 - 8 * lane - x;
                        s_digit[1] = need - above;
                        break;
                    }
                    above += c;
                }
            }
        }
        cluster.sync();                             // every CTA has read the counts; the digit is published
        prefix = (prefix << 8) | s_digit[0];
        need = s_digit[1];
    }
    // keys above `prefix` all stay, `need` of those equal to it (in index order)
    uint32_t gt = 0, eq = 0;
    for (int tw = w0; tw < w1; tw += 128) {
        uint32_t k[4];
#pragma unroll
        for (int e = 0; e < 4; e++) k[e] = tw + 32 * e + lane < w1 ? key_of(tw + 32 * e + lane) : 0u;   // (0: no row's)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            gt += k[e] > prefix;
            eq += k[e] == prefix && k[e];
        }
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        s_warp[warp][0] = gt;
        s_warp[warp][1] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t x = 0, y = 0;
        for (int w = 0; w < kSelWarps; w++) {
            x += s_warp[w][0];
            y += s_warp[w][1];
        }
        s_cta[0] = x;
        s_cta[1] = y;
    }
    cluster.sync();
    uint32_t at = 0, eq_before = 0;                 // kept rows, border keys before this warp
    for (int r = 0; r < rank; r++) {
        const uint32_t *o = cluster.map_shared_rank(s_cta, r);
        at += o[0];
        eq_before += o[1];
    }
    for (int w = 0; w < warp; w++) {
        at += s_warp[w][0];
        eq_before += s_warp[w][1];
    }
    // this CTA's kept rows [c0, c1)
    uint32_t c0 = 0, c_eq = 0;
    for (int r = 0; r < rank; r++) {
        const uint32_t *o = cluster.map_shared_rank(s_cta, r);
        c0 += o[0];
        c_eq += o[1];
    }
    const uint32_t c1 = min(c0 + s_cta[0] + min(c_eq + s_cta[1], need), (uint32_t)a.keep);
    c0 += min(c_eq, need);
    at += min(eq_before, need);
    cluster.sync();                                 // no CTA leaves while its counts may be read
    const unsigned below = (1u << lane) - 1u;
    for (int tw = w0; tw < w1; tw += 128) {
        uint32_t k[4];
#pragma unroll
        for (int e = 0; e < 4; e++) k[e] = tw + 32 * e + lane < w1 ? key_of(tw + 32 * e + lane) : 0u;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int t = tw + 32 * e + lane;
            const bool in = t < w1;
            const unsigned eqs = __ballot_sync(0xffffffffu, in && k[e] == prefix);
            const bool take = in && (k[e] > prefix || (k[e] == prefix && eq_before + (uint32_t)__popc(eqs & below) < need));
            const unsigned takes = __ballot_sync(0xffffffffu, take);
            const uint32_t to = at + (uint32_t)__popc(takes & below);
            if (take && to < (uint32_t)a.keep) kept[to] = t;
            at += (uint32_t)__popc(takes);
            eq_before += (uint32_t)__popc(eqs);
        }
    }
    gather_scores<kSelThreads>(c0, c1, src, kept, dst);
}

struct MoveArgs {
    uint8_t *pool;
    int64_t num_pages;
    int P, log2P, B, Hkv;
    int64_t slab;
    const int32_t *block_table, *new_block_table;
    int max_pages, new_max_pages, keep;
    const int32_t *kept, *new_lens;
    int dtype;
    unsigned *err;
};

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(MoveArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int groups = (a.keep + 15) / 16;
    const int64_t id = (int64_t)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
    if (id >= (int64_t)a.B * a.Hkv * groups) return;
    const int seg = (int)(id / groups), i0 = (int)(id % groups) * 16;
    const int b = seg / a.Hkv, h = seg % a.Hkv;
    const int rows = min(16, __ldcg(a.new_lens + b) - i0);   // rows of this group that exist
    if (rows <= 0) return;
    const int col = i0 >> a.log2P;
    int64_t page = -1;
    if (col < a.new_max_pages) page = a.new_block_table[(int64_t)b * a.new_max_pages + col];
    if (page < 0 || page >= a.num_pages) {
        if (lane == 0) flag_error(a.err, kErrPage);
        return;
    }
    // lane r < 16 finds the source of row r: its group's address and row (-1: flagged, not moved)
    int64_t src = -1;
    if (lane < rows) {
        const int t = __ldcg(a.kept + (int64_t)seg * a.keep + i0 + lane);
        const int64_t pg = a.block_table[(int64_t)b * a.max_pages + (t >> a.log2P)];
        if (pg < 0 || pg >= a.num_pages) flag_error(a.err, kErrPage);
        else src = (pg << a.log2P) + (t & (a.P - 1));
    }
    const bool fp8 = a.dtype == NVFP4KV_DTYPE_FP8_E4M3;
    const int bytes = fp8 ? 4096 : 2304;
    auto group_of = [&](int64_t slot) {
        const int row = (int)(slot & (a.P - 1));
        return a.pool + ((slot >> a.log2P) * a.Hkv + h) * a.slab + (row >> 4) * bytes;
    };
    uint8_t *dst = a.pool + (page * a.Hkv + h) * a.slab + ((i0 & (a.P - 1)) >> 4) * bytes;
    if (fp8) {   // K 128 bytes a row, then V: 8 chunks of 16 bytes, four rows at a time
#pragma unroll
        for (int x = 0; x < 4; x++) {
            const int r = 4 * x + (lane >> 3), ch = (lane & 7) * 16;
            const int64_t s = __shfl_sync(0xffffffffu, src, r);
            if (s < 0) continue;
            const uint8_t *from = group_of(s) + (s & 15) * 128 + ch;
            const uint4 k = *reinterpret_cast<const uint4 *>(from), v = *reinterpret_cast<const uint4 *>(from + 2048);
            *reinterpret_cast<uint4 *>(dst + r * 128 + ch) = k;
            *reinterpret_cast<uint4 *>(dst + 2048 + r * 128 + ch) = v;
        }
        return;
    }
    // codes: 4 chunks of 16 bytes a row, eight rows at a time, K and V; all loads first
    uint4 k[2], v[2];
    int64_t s[2];
#pragma unroll
    for (int x = 0; x < 2; x++) {
        const int r = 8 * x + (lane >> 2), ch = (lane & 3) * 16;
        s[x] = __shfl_sync(0xffffffffu, src, r);
        if (s[x] < 0) continue;
        const uint8_t *from = group_of(s[x]) + (s[x] & 15) * 64 + ch;
        k[x] = *reinterpret_cast<const uint4 *>(from);
        v[x] = *reinterpret_cast<const uint4 *>(from + 1152);
    }
    // K scales: lane r < 16 its row's 8 bytes.  V scales lie block-major: lane (blk, q) gathers rows 4q .. 4q + 3
    uint2 ks = make_uint2(0, 0);
    if (src >= 0) ks = *reinterpret_cast<const uint2 *>(group_of(src) + 1024 + (src & 15) * 8);
    uint8_t vs[4];
    bool ok[4];
    const int blk = lane >> 2, q = lane & 3;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const int64_t sr = __shfl_sync(0xffffffffu, src, 4 * q + e);
        ok[e] = sr >= 0;
        if (ok[e]) vs[e] = group_of(sr)[2176 + blk * 16 + (sr & 15)];
    }
#pragma unroll
    for (int x = 0; x < 2; x++) {
        const int r = 8 * x + (lane >> 2), ch = (lane & 3) * 16;
        if (s[x] < 0) continue;
        *reinterpret_cast<uint4 *>(dst + r * 64 + ch) = k[x];
        *reinterpret_cast<uint4 *>(dst + 1152 + r * 64 + ch) = v[x];
    }
    if (src >= 0) *reinterpret_cast<uint2 *>(dst + 1024 + lane * 8) = ks;
    uint8_t *vd = dst + 2176 + blk * 16 + 4 * q;
    if (ok[0] && ok[1] && ok[2] && ok[3]) {
        *reinterpret_cast<uchar4 *>(vd) = make_uchar4(vs[0], vs[1], vs[2], vs[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (ok[e]) vd[e] = vs[e];
    }
}

}  // namespace

cudaError_t launch_evict(const nvfp4kv_cache &c, const float *scores, int64_t score_stride, int batch,
                         const int32_t *block_table, int max_pages, const int32_t *seq_lens,
                         const int32_t *new_block_table, int new_max_pages, int keep, int recent, int sink,
                         int32_t *new_lens, int32_t *kept, float *new_scores, int64_t new_score_stride, unsigned *err,
                         cudaStream_t stream) {
    static std::mutex mu;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::unique_lock<std::mutex> lock(mu);
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&select_kernel<false>),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyCache * 4);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&select_kernel<true>),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyCache * 4);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&select_one_kernel<kOneLarge>),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kOneRows * 4);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    lock.unlock();
    SelectArgs a;
    a.scores = scores;
    a.score_stride = score_stride;
    a.B = batch;
    a.Hkv = c.num_kv_heads;
    a.seq_lens = seq_lens;
    const int64_t table = (int64_t)max_pages * c.page_size;
    a.cap = table < score_stride ? table : score_stride;
    a.keep = keep;
    a.recent = recent;
    a.sink = sink;
    a.new_lens = new_lens;
    a.kept = kept;
    a.new_scores = new_scores;
    a.new_score_stride = new_score_stride;
    a.err = err;
    const int64_t segs = (int64_t)batch * c.num_kv_heads;
    const bool one = a.cap <= kOneRows;
    // CTAs a segment: enough to fill the GPU when there are few segments, none with less than 1,024 rows at hand
    int cluster = 1;
    while (cluster < kMaxCluster && segs * cluster < kTargetCtasSel && a.cap >= 2048 * (int64_t)cluster) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster, (unsigned)segs, 1);
    cfg.blockDim = dim3(kSelThreads);
    const int64_t part = ceil_div64(a.cap, cluster);
    cfg.dynamicSmemBytes = (size_t)(part < kKeyCache ? part : kKeyCache) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void *args[] = {&a};
    const void *fn = part > kKeyCache ? reinterpret_cast<const void *>(&select_kernel<true>)
                                      : reinterpret_cast<const void *>(&select_kernel<false>);
    if (one) {
        const bool small = a.cap <= kOneSmallRows;
        fn = small ? reinterpret_cast<const void *>(&select_one_kernel<kOneSmall>)
                   : reinterpret_cast<const void *>(&select_one_kernel<kOneLarge>);
        cfg.gridDim = dim3((unsigned)segs);
        cfg.blockDim = dim3(small ? kOneSmall : kOneLarge);
        cfg.dynamicSmemBytes = ((size_t)a.cap + 3) / 4 * 16;
        cfg.numAttrs = 1;
    }
    e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e != cudaSuccess) return e;

    MoveArgs m;
    m.pool = static_cast<uint8_t *>(c.pool);
    m.num_pages = c.num_pages;
    m.P = c.page_size;
    m.log2P = __builtin_ctz((unsigned)c.page_size);
    m.B = batch;
    m.Hkv = c.num_kv_heads;
    m.slab = (int64_t)(c.dtype == NVFP4KV_DTYPE_NVFP4 ? 144 : 256) * c.page_size;
    m.block_table = block_table;
    m.new_block_table = new_block_table;
    m.max_pages = max_pages;
    m.new_max_pages = new_max_pages;
    m.keep = keep;
    m.kept = kept;
    m.new_lens = new_lens;
    m.dtype = c.dtype;
    m.err = err;
    const int64_t warps = segs * ((keep + 15) / 16);
    void *margs[] = {&m};
    return launch_pdl(reinterpret_cast<const void *>(&move_kernel), (unsigned)ceil_div64(warps, kMoveThreads / 32),
                      kMoveThreads, 0, stream, margs);
}

}  // namespace nvfp4kv
