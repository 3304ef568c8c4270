// rope_append.cu -- head norms, position rotation and the quantise-append of K and V in one pass.
//
// Per token and head x[128] of Q and K, with a weight w (or 1) and the token's table row (c, s):
//   r = 1 / sqrt(mean(x^2) + eps)  (1 without norms),   u = x w,
//   y_a = r (u_a c - u_b s),  y_b = r (u_b c + u_a s)   for each rotated pair (a, b),  y = r u elsewhere,
// rounded to BF16 once (a user who rotates first hands such a row to the append).  Q goes to q_out,
// K to the pool like V, which is not touched before it is quantised (quantize.cuh: the rounding of the
// exact quotients).  The rotated K leaves the kernel quantised alone: a chunk attention that takes
// the chunk's own BF16 rows needs them rotated by its caller.
//
// Bound by bandwidth: a token reads (Hq + 2 Hkv) 256 bytes and writes Hq 256 + Hkv 144.
// Eight threads hold a row, 16 values each: eight of the first rotated half and their eight
// partners (or, for adjacent pairs and behind the rotated values, one block of the format), so
// a thread needs eight cosines and sines.  Four or eight rows of one kind of one token are a
// warp's unit; Q's weights are multiplied into the cosines and sines, and its rows go through
// packed FP32 operations.  Measured, cold caches, a call alone: 32,768 tokens of 64 + 8 heads with norms 270 us (4.7
// TB/s, 69% of the copy bandwidth: 5,100 warp instructions a token at half the issue slots, the warps waiting for
// memory), the same to an FP8 pool 258, with 64 of 128 values rotated 282; 5,003 of 40 + 8 with norms, three axes and
// tensor scales 50 us, 2,048 of 32 + 2 without norms 20, 8 tokens 6.3 (latency).
//
// K's rounding to BF16 decides the codes: a value on the other side of a BF16 border may
// move a block's scale.  So K's FP32 value is rounded twice, at both ends of its error bound,
// and where they differ for some value of the warp (about 1 warp in 25, 1 in 8 with norms) its rows are formed
// again from two floats: products and sums with their rounding errors (fused multiply-adds,
// Knuth's two-sum), the sum of squares and the reciprocal root as well, and the BF16 rounding
// breaks ties by the low part: the rounding of the exact value up to a relative 2^-40 of
// the pair's larger product (of one above 2^-100, and of rows whose mean square plus eps is: below, FP32's
// subnormals lose the low parts).  Q is formed in FP32 (a value within 2^-21 of a tie may round to the other
// neighbour).
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "quantize.cuh"

namespace nvfp4kv {

namespace {

struct RopeArgs {
    uint8_t *pool;
    int64_t num_slots, slab;
    int P, log2P, Hkv, Hq;
    const uint4 *q, *k, *v;
    uint4 *q_out;
    int64_t q_stride16, kv_stride16, out_stride16;   // token strides in 16-byte units
    int64_t num_tokens;
    const int32_t *positions;                        // [axes][num_tokens]
    const float *table;                              // [num_positions][rot]: cos | sin
    int64_t num_positions;
    int rot, adjacent, sec1, sec2;                   // pairs < sec1: axis 0, < sec2: axis 1, else axis 2
    const uint4 *wq, *wk;                            // BF16 [128] or nullptr
    float eps;
    const int64_t *slots;
    float gk, gv;
    int dtype;
    unsigned *err;
};

constexpr int kThreadsR = 256;

struct Pair {
    float hi, lo;
};

// a + b = hi + lo exactly
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}

constexpr float kInfR = __builtin_huge_valf();

// hi + lo (lo small beside hi) rounded to BF16, ties of hi broken by lo; hi alone where lo is zero (a zero keeps its
// sign) or hi no finite number
__device__ __forceinline__ uint32_t bf16_of_pair(float hi, float lo) {
    if (lo == 0.0f || !(fabsf(hi) < kInfR)) return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(hi));
    const float t = __fadd_rn(hi, lo), rest = __fsub_rn(lo, __fsub_rn(t, hi));
    uint32_t b = __float_as_uint(t);
    if ((b & 0xffffu) == 0x8000u && rest != 0.0f) b += (rest > 0.0f) == (t > 0.0f) ? 1u : 0xffffffffu;
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(b)));
}

// 1 / sqrt(ssq / 128 + eps) as two floats: the hardware's estimate and one Newton step
// whose residual 1 - m r^2 is formed exactly up to 2^-44.
__device__ __forceinline__ Pair root(Pair ssq, float eps) {
    if (ssq.hi == kInfR) return {0.0f, 0.0f};
    const Pair m0 = two_sum(ssq.hi * 0.0078125f, eps);
    const float lo = m0.lo + ssq.lo * 0.0078125f;
    const float m = m0.hi + lo, ml = lo - (m - m0.hi);
    const float r = rsqrtf(m), t = __fmul_rn(r, r), te = __fmaf_rn(r, r, -t);
    const float e = __fmaf_rn(-ml, t, __fmaf_rn(-m, te, __fmaf_rn(-m, t, 1.0f)));
    return {r, 0.5f * r * e};
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ float low2(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float high2(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t bf16_pair(uint32_t w) { return pack2(bf16_lo(w), bf16_hi(w)); }

__device__ __forceinline__ void words(const uint4 &x, uint32_t (&w)[4]) { w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w; }

constexpr int kWarpsR = kThreadsR / 32;

// Where a thread's 16 values of a rotated row lie: chunk ca of eight in the first rotated half and its partner cb,
// or the two chunks of block blk.
struct Place {
    bool turned, split;
    int half8, ca, cb;    // half8: chunks of half the rotated values (even)
};

template <bool kAdj>
__device__ __forceinline__ Place place_of(const RopeArgs &a, int blk) {
    Place p;
    p.half8 = a.rot >> 4;
    p.turned = blk < p.half8;
    p.split = p.turned && !kAdj;
    p.ca = p.split ? blk : 2 * blk;
    p.cb = p.split ? blk + p.half8 : 2 * blk + 1;
    return p;
}

__device__ __forceinline__ uint4 weight_chunk(const uint4 *w, int chunk) {
    return w ? __ldg(w + chunk) : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);   // ones
}

// Q: y = x p + (its partner) m, for the pairs of values of the chunks a and b.
struct Turn {
    uint64_t pa[4], ma[4], pb[4], mb[4];
};

template <bool kAdj>
__device__ __forceinline__ void make_turn(const RopeArgs &a, const float (&c)[8], const float (&s)[8], const uint32_t (&wa)[4],
                                          const uint32_t (&wb)[4], Turn &u) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint64_t ua = bf16_pair(wa[i]), ub = bf16_pair(wb[i]);
        if (kAdj) {
            const float c0 = c[i], c1 = c[4 + i], s0 = s[i], s1 = s[4 + i];
            u.pa[i] = mul_pair(ua, pack2(c0, c0));
            u.ma[i] = mul_pair(pack2(high2(ua), low2(ua)), pack2(-s0, s0));
            u.pb[i] = mul_pair(ub, pack2(c1, c1));
            u.mb[i] = mul_pair(pack2(high2(ub), low2(ub)), pack2(-s1, s1));
        } else {
            const uint64_t cc = pack2(c[2 * i], c[2 * i + 1]), ss = pack2(s[2 * i], s[2 * i + 1]);
            u.pa[i] = mul_pair(ua, cc);
            u.ma[i] = mul_pair(ub, pack2(-s[2 * i], -s[2 * i + 1]));
            u.pb[i] = mul_pair(ub, cc);
            u.mb[i] = mul_pair(ua, ss);
        }
    }
}

// The eight threads of a row call it together (as do the four rows of the warp).  Behind the rotation the partner is
// multiplied by a sine of zero, which adds nothing while the row is finite: a row whose norm is not, and one without a
// norm, goes without.
template <bool kAdj>
__device__ __forceinline__ void turn_q(const RopeArgs &a, bool turned, const Turn &u, uint4 &xa, uint4 &xb) {
    uint32_t va[4], vb[4], ya[4], yb[4];
    words(xa, va);
    words(xb, vb);
    float r = 1.0f;
    if (a.wq) {
        uint64_t q = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint64_t x = bf16_pair(va[i]), z = bf16_pair(vb[i]);
            q = fma_pair(z, z, fma_pair(x, x, q));
        }
        float sum = low2(q) + high2(q);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        r = rsqrtf(fmaf(sum, 0.0078125f, a.eps));
    }
    auto rounded = [&](uint64_t y) {
        if (a.wq) y = mul_pair(y, pack2(r, r));
        return f32x2_to_bf16x2(high2(y), low2(y));
    };
    if (!turned && !(a.wq && r > 0.0f)) {
        if (!a.wq) return;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            ya[i] = rounded(mul_pair(bf16_pair(va[i]), u.pa[i]));
            yb[i] = rounded(mul_pair(bf16_pair(vb[i]), u.pb[i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint64_t x = bf16_pair(va[i]), z = bf16_pair(vb[i]);
            const uint64_t px = kAdj ? pack2(bf16_hi(va[i]), bf16_lo(va[i])) : z;
            const uint64_t pz = kAdj ? pack2(bf16_hi(vb[i]), bf16_lo(vb[i])) : x;
            ya[i] = rounded(fma_pair(x, u.pa[i], mul_pair(px, u.ma[i])));
            yb[i] = rounded(fma_pair(z, u.pb[i], mul_pair(pz, u.mb[i])));
        }
    }
    xa = make_uint4(ya[0], ya[1], ya[2], ya[3]);
    xb = make_uint4(yb[0], yb[1], yb[2], yb[3]);
}

// K: the chunks' exact values rounded to BF16, then exchanged so that the thread holds a whole block; returns which.
template <bool kAdj>
__device__ __forceinline__ int turn_k(const RopeArgs &a, const Place &p, int blk, const float (&c)[8], const float (&s)[8],
                                      const uint32_t (&wa)[4], const uint32_t (&wb)[4], uint4 &xa, uint4 &xb) {
    uint32_t va[4], vb[4], ya[4], yb[4];
    words(xa, va);
    words(xb, vb);
    // FP32: y = r (u c + z s) is off by at most 2^-24 (|z s| + |y|), and with a norm by 2^-20.9 |y| more (a sum of
    // squares of nine steps, 2^-21.8 in the root, its Newton step, the product); a rounding of the ends is allowed for.
    uint32_t differ = 0;
    {
        float r = 1.0f, dm = 0x1p-23f, dy = 0x1.2p-23f;
        if (a.wk) {
            uint64_t qa = 0, qb = 0;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint64_t x = bf16_pair(va[i]), z = bf16_pair(vb[i]);
                qa = fma_pair(x, x, qa);
                qb = fma_pair(z, z, qb);
            }
            float sum = (low2(qa) + high2(qa)) + (low2(qb) + high2(qb));
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const float m = fmaf(sum, 0.0078125f, a.eps), r0 = rsqrtf(m);
            r = m == kInfR ? 0.0f : fmaf(0.5f * r0, fmaf(-m * r0, r0, 1.0f), r0);
            dm *= r;
            dy = 0x1.6p-21f;
        }
        auto ends = [&](uint64_t y, float e0, float e1) {
            const uint32_t lo = f32x2_to_bf16x2(high2(y) - e1, low2(y) - e0), hi = f32x2_to_bf16x2(high2(y) + e1, low2(y) + e0);
            differ |= lo ^ hi;
            return lo;
        };
        auto both = [&](uint64_t u, uint64_t cc, uint64_t z, uint64_t ss) {
            const uint64_t m = mul_pair(z, ss);
            uint64_t y = fma_pair(u, cc, m);
            if (a.wk) y = mul_pair(y, pack2(r, r));
            return ends(y, fmaf(fabsf(low2(m)), dm, fabsf(low2(y)) * dy), fmaf(fabsf(high2(m)), dm, fabsf(high2(y)) * dy));
        };
        if (p.turned) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint64_t ua = mul_pair(bf16_pair(va[i]), bf16_pair(wa[i])), ub = mul_pair(bf16_pair(vb[i]), bf16_pair(wb[i]));
                if (kAdj) {
                    ya[i] = both(ua, pack2(c[i], c[i]), pack2(high2(ua), low2(ua)), pack2(-s[i], s[i]));
                    yb[i] = both(ub, pack2(c[4 + i], c[4 + i]), pack2(high2(ub), low2(ub)), pack2(-s[4 + i], s[4 + i]));
                } else {
                    ya[i] = both(ua, pack2(c[2 * i], c[2 * i + 1]), ub, pack2(-s[2 * i], -s[2 * i + 1]));
                    yb[i] = both(ub, pack2(c[2 * i], c[2 * i + 1]), ua, pack2(s[2 * i], s[2 * i + 1]));
                }
            }
        } else if (a.wk) {                      // (no partner: see turn_q)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint64_t y = mul_pair(mul_pair(bf16_pair(va[i]), bf16_pair(wa[i])), pack2(r, r));
                const uint64_t z = mul_pair(mul_pair(bf16_pair(vb[i]), bf16_pair(wb[i])), pack2(r, r));
                ya[i] = ends(y, fabsf(low2(y)) * dy, fabsf(high2(y)) * dy);
                yb[i] = ends(z, fabsf(low2(z)) * dy, fabsf(high2(z)) * dy);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) ya[i] = va[i], yb[i] = vb[i];
        }
    }
    if (__any_sync(0xffffffffu, differ != 0)) {
        Pair r = {1.0f, 0.0f};
        if (a.wk) {
            Pair q = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float v[4] = {bf16_lo(va[i]), bf16_hi(va[i]), bf16_lo(vb[i]), bf16_hi(vb[i])};
#pragma unroll
                for (int e = 0; e < 4; e++) {                     // (a BF16 number's square is exact)
                    const Pair n = two_sum(q.hi, __fmul_rn(v[e], v[e]));
                    q = {n.hi, q.lo + n.lo};
                }
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) {
                const float h = __shfl_xor_sync(0xffffffffu, q.hi, d), lo = __shfl_xor_sync(0xffffffffu, q.lo, d);
                const Pair n = two_sum(q.hi, h);
                q = {n.hi, (q.lo + lo) + n.lo};
            }
            r = root(q, a.eps);
        }
        // r (u cc + z ss) rounded to BF16, u and z exact products of 16 bits
        auto exact = [&](float u, float cc, float z, float ss) {
            Pair d = {u, 0.0f};
            if (p.turned) {
                const float h = __fmul_rn(u, cc), k = __fmul_rn(z, ss);
                const Pair n = two_sum(h, k);
                d = {n.hi, n.lo + (__fmaf_rn(u, cc, -h) + __fmaf_rn(z, ss, -k))};
            }
            if (a.wk) {
                const float h = __fmul_rn(d.hi, r.hi);
                d = {h, __fmaf_rn(d.lo, r.hi, __fmaf_rn(d.hi, r.lo, __fmaf_rn(d.hi, r.hi, -h)))};
            }
            return bf16_of_pair(d.hi, d.lo);
        };
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float a0 = bf16_lo(va[i]) * bf16_lo(wa[i]), a1 = bf16_hi(va[i]) * bf16_hi(wa[i]);
            const float b0 = bf16_lo(vb[i]) * bf16_lo(wb[i]), b1 = bf16_hi(vb[i]) * bf16_hi(wb[i]);
            if (kAdj) {
                ya[i] = exact(a0, c[i], a1, -s[i]) | (exact(a1, c[i], a0, s[i]) << 16);
                yb[i] = exact(b0, c[4 + i], b1, -s[4 + i]) | (exact(b1, c[4 + i], b0, s[4 + i]) << 16);
            } else {
                ya[i] = exact(a0, c[2 * i], b0, -s[2 * i]) | (exact(a1, c[2 * i + 1], b1, -s[2 * i + 1]) << 16);
                yb[i] = exact(b0, c[2 * i], a0, s[2 * i]) | (exact(b1, c[2 * i + 1], a1, s[2 * i + 1]) << 16);
            }
        }
    }
    // Two threads of a half-split pair of chunks exchange one each: the even one quantises the block of the
    // first half, the odd one that of the second.
    const bool odd = blk & 1;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? ya[i] : yb[i], 1);
        if (p.split) {
            if (odd) ya[i] = other;
            else yb[i] = other;
        }
    }
    xa = make_uint4(ya[0], ya[1], ya[2], ya[3]);
    xb = make_uint4(yb[0], yb[1], yb[2], yb[3]);
    return !p.split ? blk : odd ? (blk - 1 + p.half8) >> 1 : blk >> 1;
}

// A thread's cosines and sines from a row of the table (cosines, then sines) of its pair groups x (two of four pairs).
__device__ __forceinline__ void take4(float (&v)[8], int i, const float4 &x) {
    v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
}

__device__ __forceinline__ int axis_of(const RopeArgs &a, int pair) { return pair < a.sec1 ? 0 : pair < a.sec2 ? 1 : 2; }
__device__ __forceinline__ int axes_of(const RopeArgs &a) { return a.sec1 >= kHeadDim ? 1 : a.sec2 >= kHeadDim ? 2 : 3; }

// Few tokens: a warp takes four rows of one kind of a token, everything straight from global memory.
template <bool kUnitScale, bool kAdj>
__global__ void __launch_bounds__(kThreadsR) rope_append_kernel(RopeArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t id = (int64_t)blockIdx.x * kWarpsR + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, blk = lane & 7, g = lane >> 3;
    const int nq = (a.Hq + 3) / 4, nk = (a.Hkv + 3) / 4;
    const int64_t t = id / (nq + 2 * nk);
    const int sub = (int)(id - t * (nq + 2 * nk));
    if (t >= a.num_tokens) return;                            // (the whole warp)
    const bool is_q = sub < nq, is_k = !is_q && sub < nq + nk;
    Place p = place_of<kAdj>(a, blk);
    if (!is_q && !is_k) p.turned = p.split = false, p.ca = 2 * blk, p.cb = 2 * blk + 1;
    const int row = 4 * (is_q ? sub : is_k ? sub - nq : sub - nq - nk) + g, nrows = is_q ? a.Hq : a.Hkv;
    const uint4 *base = (is_q ? a.q + t * a.q_stride16 : (is_k ? a.k : a.v) + t * a.kv_stride16) + row * 16;
    uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
    if (row < nrows) {
        xa = __ldg(base + p.ca);
        xb = __ldg(base + p.cb);
    }
    const int64_t slot = __ldg(a.slots + t);
    bool ok = true;                                           // (all of the token's positions: any warp skips it)
    if (a.rot > 0) {
        for (int x = 0; x < axes_of(a); x++) {
            const int32_t pos = __ldg(a.positions + x * a.num_tokens + t);
            ok = ok && pos >= 0 && pos < a.num_positions;
        }
    }
    if (sub == 0 && lane == 0) {
        if (!ok) flag_error(a.err, kErrPosition);
        if (slot >= a.num_slots) flag_error(a.err, kErrSlot);
    }
    if (!ok) return;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; i++) c[i] = 1.f, s[i] = 0.f;
    if (p.turned) {
#pragma unroll
        for (int i = 0; i < 2; i++) {                         // (four pairs lie in one section)
            const int pair = 8 * blk + 4 * i;
            const int32_t pos = __ldg(a.positions + axis_of(a, pair) * a.num_tokens + t);
            const float4 *at = reinterpret_cast<const float4 *>(a.table + (int64_t)pos * a.rot + pair);
            take4(c, i, __ldg(at));
            take4(s, i, __ldg(at + (a.rot >> 3)));
        }
    }
    if (is_q) {
        uint32_t wa[4], wb[4];
        words(weight_chunk(a.wq, p.ca), wa);
        words(weight_chunk(a.wq, p.cb), wb);
        Turn u;
        make_turn<kAdj>(a, c, s, wa, wb, u);
        turn_q<kAdj>(a, p.turned, u, xa, xb);
        if (row < nrows) {
            uint4 *dst = a.q_out + t * a.out_stride16 + row * 16;
            dst[p.ca] = xa;
            dst[p.cb] = xb;
        }
        return;
    }
    if (slot < 0 || slot >= a.num_slots) return;
    int at = blk;
    if (is_k) {
        uint32_t wa[4], wb[4];
        words(weight_chunk(a.wk, p.ca), wa);
        words(weight_chunk(a.wk, p.cb), wb);
        at = turn_k<kAdj>(a, p, blk, c, s, wa, wb, xa, xb);
    }
    if (row < nrows)
        store_block_values<kUnitScale, true>(a.pool + ((slot >> a.log2P) * a.Hkv + row) * a.slab, a.dtype, (int)(slot & (a.P - 1)),
                                             !is_k, at, xa, xb, is_k ? a.gk : a.gv, l2_policy_evict_last());
}

// Many tokens: persistent CTAs.  One warp copies whole tokens (rows of Q, K and V, the pieces of the table) into a ring
// in shared memory, eight warps work on four rows at a time from there.  The direct form's loads, a chain of position,
// table row and use, leaves DRAM idle: 32,768 tokens of 64 + 8 heads with norms take it 372 us, the ring 270.
constexpr int kThreadsS = kThreadsR + 32;
constexpr int kStreamBytes = 110 * 1024;          // of a CTA's ring, two CTAs an SM
constexpr int kMaxStages = 8, kMaxTps = 32;
constexpr uint32_t kWaitLimitR = 1u << 22;

struct StreamPlan {
    int tps, stages;       // tokens a stage, stages
    int token_bytes;       // rows and table pieces of a token
};

struct StreamMisc {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int64_t slot[kMaxStages][kMaxTps];            // -1: K and V are skipped; kNoToken: all of it
    int abort;
};
constexpr int64_t kNoToken = -2;

// kAll: all 128 values are rotated, a form of its own for adjacent pairs (32,768 tokens of 64 + 8 heads with norms: 285 us
// without it, 271 so; half-split pairs 270 without, 304 so).
template <bool kUnitScale, bool kAdj, bool kAll>
__global__ void __launch_bounds__(kThreadsS, 2) rope_stream_kernel(RopeArgs a, StreamPlan plan) {
    extern __shared__ __align__(128) uint8_t smem[];
    StreamMisc &m = *reinterpret_cast<StreamMisc *>(smem + plan.stages * plan.tps * plan.token_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < plan.stages; i++) {
            mbar_init(&m.full[i], 1);
            mbar_init(&m.empty[i], kWarpsR);
        }
        m.abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    volatile int *abort_flag = &m.abort;
    const int64_t tiles = (a.num_tokens + plan.tps - 1) / plan.tps;
    const int q_bytes = a.Hq * 256, kv_bytes = a.Hkv * 256;
    int st = 0;
    uint32_t ph = 0;
    bool good = true;
    if (warp == kWarpsR) {
        // ---------------- the copying warp: lane i < tps takes token i of a stage
        const int axes = a.rot > 0 ? axes_of(a) : 0;
        int32_t pos[3] = {0, 0, 0};
        int64_t slot = 0;
        auto fetch = [&](int64_t tile) {
            const int64_t t = tile * plan.tps + lane;
            if (lane >= plan.tps || t >= a.num_tokens) return;
            for (int x = 0; x < 3; x++)
                if (x < axes) pos[x] = __ldg(a.positions + x * a.num_tokens + t);
            slot = __ldg(a.slots + t);
        };
        fetch(blockIdx.x);
        int64_t done = 0;
        for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, done++) {
            if (done >= plan.stages) good = __all_sync(0xffffffffu, mbar_wait_bounded(&m.empty[st], ph ^ 1u, kWaitLimitR, abort_flag));
            if (!good) break;
            const int64_t t = tile * plan.tps + lane;
            const bool there = lane < plan.tps && t < a.num_tokens;
            bool ok = there;
#pragma unroll
            for (int x = 0; x < 3; x++) ok = ok && (x >= axes || (pos[x] >= 0 && pos[x] < a.num_positions));
            if (there && !ok) flag_error(a.err, kErrPosition);
            if (there && slot >= a.num_slots) flag_error(a.err, kErrSlot);
            const bool write = ok && slot >= 0 && slot < a.num_slots;
            if (lane < plan.tps) m.slot[st][lane] = !ok ? kNoToken : write ? slot : -1;
            const uint32_t bytes = ok ? q_bytes + 4 * a.rot + (write ? 2 * kv_bytes : 0) : 0;
            const uint32_t total = __reduce_add_sync(0xffffffffu, bytes);
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&m.full[st], total);
            __syncwarp();
            if (ok) {
                uint8_t *dst = smem + (st * plan.tps + lane) * plan.token_bytes;
                if (q_bytes) bulk_g2s(dst, a.q + t * a.q_stride16, q_bytes, &m.full[st]);
                if (write) {
                    bulk_g2s(dst + q_bytes, a.k + t * a.kv_stride16, kv_bytes, &m.full[st]);
                    bulk_g2s(dst + q_bytes + kv_bytes, a.v + t * a.kv_stride16, kv_bytes, &m.full[st]);
                }
                dst += q_bytes + 2 * kv_bytes;
                for (int x = 0; x < axes; x++) {              // the pairs of axis x: cosines and sines
                    const int first = x == 0 ? 0 : x == 1 ? a.sec1 : a.sec2;
                    const int end = min(a.rot / 2, x == 0 ? a.sec1 : x == 1 ? a.sec2 : kHeadDim);
                    if (end <= first) continue;
                    const float *row = a.table + (int64_t)pos[x] * a.rot;
                    if (axes == 1) {
                        bulk_g2s(dst, row, 4 * a.rot, &m.full[st]);
                    } else {
                        bulk_g2s(dst + 4 * first, row + first, 4 * (end - first), &m.full[st]);
                        bulk_g2s(dst + 2 * a.rot + 4 * first, row + a.rot / 2 + first, 4 * (end - first), &m.full[st]);
                    }
                }
            }
            fetch(tile + gridDim.x);
            if (++st == plan.stages) st = 0, ph ^= 1u;
        }
        // no copy may still be writing when the CTA ends
        for (int64_t i = done > plan.stages ? done - plan.stages : 0; i < done; i++)
            mbar_wait_bounded(&m.full[i % plan.stages], (uint32_t)(i / plan.stages) & 1, kWaitLimitR, nullptr);
    } else {
        const int blk = lane & 7, g = lane >> 3;
        Place p = place_of<kAdj>(a, blk);
        if (kAll) p.turned = true, p.split = !kAdj;
        // A token's units: four rows of K, four of V, eight of Q.  Those of K take longest, so the warps take turns.
        const int nq = (a.Hq + 7) / 8, nk = (a.Hkv + 3) / 4, per = nq + 2 * nk;
        const uint64_t policy = l2_policy_evict_last();
        int turn = warp;
        for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            good = __all_sync(0xffffffffu, mbar_wait_bounded(&m.full[st], ph, kWaitLimitR, abort_flag));
            if (!good) break;
            const int n = (int)min((int64_t)plan.tps, a.num_tokens - tile * plan.tps);
            for (int sub = turn, i = 0;; sub += kWarpsR) {
                for (; sub >= per && i < n; i++) sub -= per;
                if (i >= n) {
                    turn = sub;                               // the next stage's units go on behind this one's
                    break;
                }
                const int64_t slot = m.slot[st][i], t = tile * plan.tps + i;
                if (slot == kNoToken || (sub < 2 * nk && slot < 0)) continue;
                const uint8_t *src = smem + (st * plan.tps + i) * plan.token_bytes;
                float c[8], s[8];
                if (sub < nk || sub >= 2 * nk) {
                    const float *table = reinterpret_cast<const float *>(src + q_bytes + 2 * kv_bytes);
#pragma unroll
                    for (int x = 0; x < 8; x++) c[x] = 1.f, s[x] = 0.f;
                    if (p.turned) {
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            take4(c, x, *reinterpret_cast<const float4 *>(table + 8 * blk + 4 * x));
                            take4(s, x, *reinterpret_cast<const float4 *>(table + (a.rot >> 1) + 8 * blk + 4 * x));
                        }
                    }
                }
                uint32_t wa[4], wb[4];                        // (from L1: registers are short)
                if (sub < 2 * nk) {
                    const bool is_k = sub < nk;
                    const int row = 4 * (is_k ? sub : sub - nk) + g;
                    uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
                    if (row < a.Hkv) {
                        const uint4 *x = reinterpret_cast<const uint4 *>(src + q_bytes + (is_k ? 0 : kv_bytes) + row * 256);
                        xa = x[is_k ? p.ca : 2 * blk];
                        xb = x[is_k ? p.cb : 2 * blk + 1];
                    }
                    int at = blk;
                    if (is_k) {
                        words(weight_chunk(a.wk, p.ca), wa);
                        words(weight_chunk(a.wk, p.cb), wb);
                        at = turn_k<kAdj>(a, p, blk, c, s, wa, wb, xa, xb);
                    }
                    if (row < a.Hkv)
                        store_block_values<kUnitScale, true>(a.pool + ((slot >> a.log2P) * a.Hkv + row) * a.slab, a.dtype,
                                                             (int)(slot & (a.P - 1)), !is_k, at, xa, xb, is_k ? a.gk : a.gv, policy);
                } else {
                    const int row = 8 * (sub - 2 * nk) + g;
                    uint4 xa[2], xb[2];
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const uint4 *x = reinterpret_cast<const uint4 *>(src + (row + 4 * e) * 256);
                        xa[e] = xb[e] = make_uint4(0, 0, 0, 0);
                        if (row + 4 * e < a.Hq) {
                            xa[e] = x[p.ca];
                            xb[e] = x[p.cb];
                        }
                    }
                    words(weight_chunk(a.wq, p.ca), wa);
                    words(weight_chunk(a.wq, p.cb), wb);
                    Turn u;
                    make_turn<kAdj>(a, c, s, wa, wb, u);
#pragma unroll
                    for (int e = 0; e < 2; e++) turn_q<kAdj>(a, p.turned, u, xa[e], xb[e]);
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        if (row + 4 * e >= a.Hq) continue;
                        uint4 *dst = a.q_out + t * a.out_stride16 + (row + 4 * e) * 16;
                        dst[p.ca] = xa[e];
                        dst[p.cb] = xb[e];
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.empty[st]);
            if (++st == plan.stages) st = 0, ph ^= 1u;
        }
    }
    if (!good) {
        if (lane == 0 && !*abort_flag) flag_error(a.err, kErrTimeout);
        *abort_flag = 1;
    }
}

constexpr int kMaxDevicesR = 64;
std::mutex g_mu_r;
int g_sms_r[kMaxDevicesR];      // 0: not set up yet

}  // namespace

cudaError_t launch_rope_append(const nvfp4kv_cache &c, const nvfp4kv_rope &rope, const void *q, int64_t q_stride,
                               void *q_out, int64_t q_out_stride, int num_q_heads, const void *k, const void *v,
                               int64_t kv_stride, int64_t num_tokens, const int32_t *positions,
                               const int64_t *slot_mapping, unsigned *err, cudaStream_t stream) {
    RopeArgs a = {};
    a.pool = static_cast<uint8_t *>(c.pool);
    a.num_slots = c.num_pages * (int64_t)c.page_size;
    a.slab = (int64_t)(c.dtype == NVFP4KV_DTYPE_NVFP4 ? 144 : 256) * c.page_size;
    a.P = c.page_size;
    a.log2P = __builtin_ctz((unsigned)c.page_size);
    a.Hkv = c.num_kv_heads;
    a.Hq = num_q_heads;
    a.q = static_cast<const uint4 *>(q);
    a.k = static_cast<const uint4 *>(k);
    a.v = static_cast<const uint4 *>(v);
    a.q_out = static_cast<uint4 *>(q_out);
    a.q_stride16 = q_stride / 8;
    a.kv_stride16 = kv_stride / 8;
    a.out_stride16 = q_out_stride / 8;
    a.num_tokens = num_tokens;
    a.positions = positions;
    a.table = rope.cos_sin;
    a.num_positions = rope.num_positions;
    a.rot = rope.rot_dim;
    a.adjacent = rope.adjacent;
    a.sec1 = rope.num_axes > 1 ? rope.sections[0] : kHeadDim;
    a.sec2 = rope.num_axes > 2 ? rope.sections[0] + rope.sections[1] : kHeadDim;
    a.wq = static_cast<const uint4 *>(rope.q_norm);
    a.wk = static_cast<const uint4 *>(rope.k_norm);
    a.eps = rope.eps;
    a.slots = slot_mapping;
    a.gk = c.k_global_scale;
    a.gv = c.v_global_scale;
    a.dtype = c.dtype;
    a.err = err;
    const bool unit = c.k_global_scale == 1.0f && c.v_global_scale == 1.0f;
    const int64_t groups = (a.Hq + 3) / 4 + 2 * ((a.Hkv + 3) / 4);
    StreamPlan plan;
    plan.token_bytes = (a.Hq + 2 * a.Hkv) * 256 + 4 * a.rot;
    plan.tps = std::max(1, std::min(kMaxTps, 16 * 1024 / plan.token_bytes));
    plan.stages = std::min(kMaxStages, (int)((kStreamBytes - sizeof(StreamMisc)) / ((size_t)plan.tps * plan.token_bytes)));
    // The ring (of two stages at least) from 18,000 groups of four rows on, a compromise: it gains earlier without norms
    // and with more rows of Q beside those of K.  Direct form and ring in us, with norms | without, adjacent pairs:
    //   64 + 8 heads   256 tokens (5,000 groups) 11.4, 12.3;   1,024 (20,000) 20.3, 20.0 | 20.3, 16.6;   2,048 31.0, 28.6 |
    //                  32.6, 24.0;   16,384 190.5, 142;   32,768 372, 270
    //   32 + 8         1,024 (12,000) 15.6, 18.7;   1,500 (18,000) 18.6, 21.8 | 18.3, 18.2;   2,048 22.5, 26.4 | 22.8, 20.8;
    //                  4,096 38.4, 39.8
    //   32 + 2         2,048 (20,000) 22.4, 21.4 | 22.3, 18.5
    //   4 + 1          1,024 (3,000) 10.1, 12.7;   4,096 (12,000) 20.4, 20.5;   6,000 (18,000) 26.0, 26.4 | 26.5, 22.6;
    //                  8,192 32.5, 30.5 | 34.5, 26.4
    if (plan.stages < 2 || num_tokens * groups < 18000) {
        void *args[] = {&a};
        const void *few[2][2] = {{reinterpret_cast<const void *>(&rope_append_kernel<false, false>),
                                  reinterpret_cast<const void *>(&rope_append_kernel<false, true>)},
                                 {reinterpret_cast<const void *>(&rope_append_kernel<true, false>),
                                  reinterpret_cast<const void *>(&rope_append_kernel<true, true>)}};
        return launch_pdl(few[unit][a.adjacent], dim3((unsigned)ceil_div64(num_tokens * groups, kWarpsR)), kThreadsR, 0, stream,
                          args);
    }
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevicesR)) e = cudaErrorInvalidDevice;
    if (e != cudaSuccess) return e;
    const void *fn[2][3] = {{reinterpret_cast<const void *>(&rope_stream_kernel<false, false, false>),
                             reinterpret_cast<const void *>(&rope_stream_kernel<false, true, false>),
                             reinterpret_cast<const void *>(&rope_stream_kernel<false, true, true>)},
                            {reinterpret_cast<const void *>(&rope_stream_kernel<true, false, false>),
                             reinterpret_cast<const void *>(&rope_stream_kernel<true, true, false>),
                             reinterpret_cast<const void *>(&rope_stream_kernel<true, true, true>)}};
    {
        std::lock_guard<std::mutex> lock(g_mu_r);
        if (!g_sms_r[dev]) {
            for (int i = 0; i < 6; i++) {
                e = cudaFuncSetAttribute(fn[i / 3][i % 3], cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes);
                if (e != cudaSuccess) return e;
            }
            e = cudaDeviceGetAttribute(&g_sms_r[dev], cudaDevAttrMultiProcessorCount, dev);
            if (e != cudaSuccess) return e;
        }
        sms = g_sms_r[dev];
    }
    void *args[] = {&a, &plan};
    const int64_t grid = std::min((int64_t)2 * sms, (num_tokens + plan.tps - 1) / plan.tps);
    return launch_pdl(fn[unit][!a.adjacent ? 0 : a.rot < kHeadDim ? 1 : 2], dim3((unsigned)grid), kThreadsS,
                      (size_t)plan.stages * plan.tps * plan.token_bytes + sizeof(StreamMisc), stream, args);
}

}  // namespace nvfp4kv
