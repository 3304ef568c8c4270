// rope_append.cu -- head norms, position rotation and the quantise-append of K and V in one pass.
//
// Per token and head x[128] of Q and K, with a weight w (or 1) and the token's table row (c, s):
//   r = 1 / sqrt(mean(x^2) + eps)  (1 without norms),   u = x w,
//   y_a = r (u_a c - u_b s),  y_b = r (u_b c + u_a s)   for each rotated pair (a, b),  y = r u elsewhere,
// rounded to BF16 once (a user who rotates first hands such a row to the append, and the
// chunk attention reads the same K).  Q goes to q_out, K to the pool like V, which is not
// touched before it is quantised (quantize.cuh: the rounding of the exact quotients).
//
// Bound by bandwidth: a token reads (Hq + 2 Hkv) 256 bytes and writes Hq 256 + Hkv 144.
// Eight threads hold a row, 16 values each: eight of the first rotated half and their eight
// partners (or, for adjacent pairs and behind the rotated values, one block of the format), so
// a thread needs eight cosines and sines.  Each warp takes rows of one kind of one token --
// 4 J rows of Q, 4 of K, 4 or 8 of V -- and loads them all first.  Q's weights are multiplied into
// the cosines and sines once a warp, and its rows go through packed FP32 operations.
//
// K's rounding to BF16 decides the codes: a value on the other side of a BF16 border may
// move a block's scale.  So K is formed from two floats: products and sums with their
// rounding errors (fused multiply-adds, Knuth's two-sum), the sum of squares and the
// reciprocal root as well, and the BF16 rounding breaks ties by the low part; it is the
// rounding of the exact value up to a relative 2^-40 of the pair's larger product.  Q is formed in FP32
// (a value within 2^-21 of a tie may round to the other neighbour).
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

// hi + lo (lo small beside hi) rounded to BF16, ties of hi broken by lo
__device__ __forceinline__ uint32_t bf16_of_pair(float hi, float lo) {
    const float t = __fadd_rn(hi, lo), rest = __fsub_rn(lo, __fsub_rn(t, hi));
    uint32_t b = __float_as_uint(t);
    if ((b & 0xffffu) == 0x8000u && rest != 0.0f) b += (rest > 0.0f) == (t > 0.0f) ? 1u : 0xffffffffu;
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(b)));
}

// 1 / sqrt(ssq / 128 + eps) as two floats: the hardware's estimate and one Newton step
// whose residual 1 - m r^2 is formed exactly up to 2^-44.
__device__ __forceinline__ Pair root(Pair ssq, float eps) {
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

// JQ: passes of four rows a warp makes over Q (and JQ > 1: two over V).
template <int JQ, bool kUnitScale>
__global__ void __launch_bounds__(kThreadsR, 2) rope_append_kernel(RopeArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int JV = JQ > 1 ? 2 : 1;
    const int64_t id = (int64_t)blockIdx.x * kWarpsR + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, blk = lane & 7, g = lane >> 3;
    const int nq = (a.Hq + 4 * JQ - 1) / (4 * JQ), nk = (a.Hkv + 3) / 4, nv = (a.Hkv + 4 * JV - 1) / (4 * JV);
    const int64_t t = id / (nq + nk + nv);
    const int sub = (int)(id - t * (nq + nk + nv));
    if (t >= a.num_tokens) return;                            // (the whole warp)
    const bool is_q = sub < nq, is_k = !is_q && sub < nq + nk;
    // The thread's two chunks of eight values: ca in the first rotated half and its partner cb, or a block's
    // (2 blk, 2 blk + 1).
    const int half8 = a.rot >> 4;                             // chunks of half the rotated values (even)
    const bool turned = is_q || is_k ? (a.adjacent ? 2 * blk < 2 * half8 : blk < half8) : false;
    const bool split = turned && !a.adjacent;
    const int ca = split ? blk : 2 * blk, cb = split ? blk + half8 : 2 * blk + 1;
    // ---- the rows
    constexpr int JM = JQ > JV ? JQ : JV;
    const int row0 = is_q ? sub * 4 * JQ : is_k ? (sub - nq) * 4 : (sub - nq - nk) * 4 * JV;
    const int nrows = is_q ? a.Hq : a.Hkv, passes = is_q ? JQ : is_k ? 1 : JV;
    const uint4 *base = is_q ? a.q + t * a.q_stride16 : (is_k ? a.k : a.v) + t * a.kv_stride16;
    uint4 xa[JM], xb[JM];
#pragma unroll
    for (int j = 0; j < JM; j++) {
        const int row = row0 + 4 * j + g;
        xa[j] = xb[j] = make_uint4(0, 0, 0, 0);
        if (j < passes && row < nrows) {
            xa[j] = __ldg(base + row * 16 + ca);
            xb[j] = __ldg(base + row * 16 + cb);
        }
    }
    const int64_t slot = is_q ? 0 : __ldg(a.slots + t);
    // ---- the positions (all of the token's: any warp skips it), and the pairs' row of the table
    bool ok = true;
    if (a.rot > 0) {
        const int axes = a.sec1 >= kHeadDim ? 1 : a.sec2 >= kHeadDim ? 2 : 3;
        for (int x = 0; x < axes; x++) {
            const int32_t pos = __ldg(a.positions + x * a.num_tokens + t);
            ok = ok && pos >= 0 && pos < a.num_positions;
        }
    }
    if (sub == 0 && lane == 0) {
        const int64_t s0 = __ldg(a.slots + t);
        if (!ok) flag_error(a.err, kErrPosition);
        if (s0 >= a.num_slots) flag_error(a.err, kErrSlot);
    }
    if (!ok) return;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; i++) c[i] = 1.f, s[i] = 0.f;
    if (turned) {
#pragma unroll
        for (int i = 0; i < 2; i++) {                         // (four pairs lie in one section)
            const int pair = 8 * blk + 4 * i, axis = pair < a.sec1 ? 0 : pair < a.sec2 ? 1 : 2;
            const int32_t pos = __ldg(a.positions + axis * a.num_tokens + t);
            const float4 *at = reinterpret_cast<const float4 *>(a.table + (int64_t)pos * a.rot + pair);
            const float4 x = __ldg(at), y = __ldg(at + (a.rot >> 3));
            c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
            s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
        }
    }
    const uint4 *weight = is_q ? a.wq : is_k ? a.wk : nullptr;
    uint32_t wa[4], wb[4];
    words(weight ? __ldg(weight + ca) : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), wa);
    words(weight ? __ldg(weight + cb) : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), wb);
    if (is_q) {
        // y = x p + (its partner) m, for the pairs of values of chunk a and chunk b
        uint64_t pa[4], ma[4], pb[4], mb[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint64_t ua = bf16_pair(wa[i]), ub = bf16_pair(wb[i]);
            if (a.adjacent) {
                const float c0 = c[i], c1 = c[4 + i], s0 = s[i], s1 = s[4 + i];
                pa[i] = mul_pair(ua, pack2(c0, c0));
                ma[i] = mul_pair(pack2(high2(ua), low2(ua)), pack2(-s0, s0));
                pb[i] = mul_pair(ub, pack2(c1, c1));
                mb[i] = mul_pair(pack2(high2(ub), low2(ub)), pack2(-s1, s1));
            } else {
                const uint64_t cc = pack2(c[2 * i], c[2 * i + 1]), ss = pack2(s[2 * i], s[2 * i + 1]);
                pa[i] = mul_pair(ua, cc);
                ma[i] = mul_pair(ub, pack2(-s[2 * i], -s[2 * i + 1]));
                pb[i] = mul_pair(ub, cc);
                mb[i] = mul_pair(ua, ss);
            }
        }
#pragma unroll
        for (int j = 0; j < JQ; j++) {
            const int row = row0 + 4 * j + g;
            uint32_t va[4], vb[4];
            words(xa[j], va);
            words(xb[j], vb);
            uint64_t ya[4], yb[4], q = 0;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint64_t x = bf16_pair(va[i]), z = bf16_pair(vb[i]);
                const uint64_t px = a.adjacent ? pack2(bf16_hi(va[i]), bf16_lo(va[i])) : z;
                const uint64_t pz = a.adjacent ? pack2(bf16_hi(vb[i]), bf16_lo(vb[i])) : x;
                ya[i] = fma_pair(x, pa[i], mul_pair(px, ma[i]));
                yb[i] = fma_pair(z, pb[i], mul_pair(pz, mb[i]));
                q = fma_pair(z, z, fma_pair(x, x, q));
            }
            if (weight) {
                float sum = low2(q) + high2(q);
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float r = rsqrtf(fmaf(sum, 0.0078125f, a.eps));
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    ya[i] = mul_pair(ya[i], pack2(r, r));
                    yb[i] = mul_pair(yb[i], pack2(r, r));
                }
            }
            if (row < nrows) {
                uint4 *dst = a.q_out + t * a.out_stride16 + row * 16;
                dst[ca] = make_uint4(f32x2_to_bf16x2(high2(ya[0]), low2(ya[0])), f32x2_to_bf16x2(high2(ya[1]), low2(ya[1])),
                                     f32x2_to_bf16x2(high2(ya[2]), low2(ya[2])), f32x2_to_bf16x2(high2(ya[3]), low2(ya[3])));
                dst[cb] = make_uint4(f32x2_to_bf16x2(high2(yb[0]), low2(yb[0])), f32x2_to_bf16x2(high2(yb[1]), low2(yb[1])),
                                     f32x2_to_bf16x2(high2(yb[2]), low2(yb[2])), f32x2_to_bf16x2(high2(yb[3]), low2(yb[3])));
            }
        }
        return;
    }
    if (slot < 0 || slot >= a.num_slots) return;
    const int64_t page = slot >> a.log2P;
    const int in_page = (int)(slot & (a.P - 1));
    const uint64_t policy = l2_policy_evict_last();           // of scale bytes, as in the plain append
    if (!is_k) {
#pragma unroll
        for (int j = 0; j < JV; j++) {
            const int row = row0 + 4 * j + g;
            if (row < nrows)
                store_block_values<kUnitScale, true>(a.pool + (page * a.Hkv + row) * a.slab, a.dtype, in_page, 1, blk, xa[j],
                                                     xb[j], a.gv, policy);
        }
        return;
    }
    const int row = row0 + g;
    uint32_t va[4], vb[4], ya[4], yb[4];
    words(xa[0], va);
    words(xb[0], vb);
    Pair r = {1.0f, 0.0f};
    if (weight) {
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
    // r (u cc + p ss) rounded to BF16, u and p exact products of 16 bits
    auto exact = [&](float u, float cc, float p, float ss) {
        Pair d = {u, 0.0f};
        if (turned) {
            const float h = __fmul_rn(u, cc), k = __fmul_rn(p, ss);
            const Pair z = two_sum(h, k);
            d = {z.hi, z.lo + (__fmaf_rn(u, cc, -h) + __fmaf_rn(p, ss, -k))};
        }
        if (weight) {
            const float h = __fmul_rn(d.hi, r.hi);
            d = {h, __fmaf_rn(d.lo, r.hi, __fmaf_rn(d.hi, r.lo, __fmaf_rn(d.hi, r.hi, -h)))};
        }
        return bf16_of_pair(d.hi, d.lo);
    };
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float a0 = bf16_lo(va[i]) * bf16_lo(wa[i]), a1 = bf16_hi(va[i]) * bf16_hi(wa[i]);
        const float b0 = bf16_lo(vb[i]) * bf16_lo(wb[i]), b1 = bf16_hi(vb[i]) * bf16_hi(wb[i]);
        if (a.adjacent) {
            ya[i] = exact(a0, c[i], a1, -s[i]) | (exact(a1, c[i], a0, s[i]) << 16);
            yb[i] = exact(b0, c[4 + i], b1, -s[4 + i]) | (exact(b1, c[4 + i], b0, s[4 + i]) << 16);
        } else {
            ya[i] = exact(a0, c[2 * i], b0, -s[2 * i]) | (exact(a1, c[2 * i + 1], b1, -s[2 * i + 1]) << 16);
            yb[i] = exact(b0, c[2 * i], a0, s[2 * i]) | (exact(b1, c[2 * i + 1], a1, s[2 * i + 1]) << 16);
        }
    }
    // Two threads of a half-split pair of chunks exchange one each: the even one quantises the block of the
    // first half, the odd one that of the second.
    const bool odd = blk & 1;
    int at = blk;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? ya[i] : yb[i], 1);
        if (split) {
            if (odd) ya[i] = other;
            else yb[i] = other;
        }
    }
    if (split) at = odd ? (blk - 1 + half8) >> 1 : blk >> 1;
    if (row < nrows)
        store_block_values<kUnitScale, true>(a.pool + (page * a.Hkv + row) * a.slab, a.dtype, in_page, 0, at,
                                             make_uint4(ya[0], ya[1], ya[2], ya[3]), make_uint4(yb[0], yb[1], yb[2], yb[3]),
                                             a.gk, policy);
}

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
    // Four rows a warp while that does not fill the GPU (two CTAs on each of 152 SMs), more beyond.
    const bool many = num_tokens * (a.Hq + 2 * a.Hkv) > 4 * 152 * 2 * kWarpsR;
    const int jq = many ? 4 : 1, jv = many ? 2 : 1;
    const int64_t warps = (a.Hq + 4 * jq - 1) / (4 * jq) + (a.Hkv + 3) / 4 + (a.Hkv + 4 * jv - 1) / (4 * jv);
    const int64_t grid = ceil_div64(num_tokens * warps, kWarpsR);
    const bool unit = c.k_global_scale == 1.0f && c.v_global_scale == 1.0f;
    void *args[] = {&a};
    const void *fn = many ? (unit ? reinterpret_cast<const void *>(&rope_append_kernel<4, true>)
                                  : reinterpret_cast<const void *>(&rope_append_kernel<4, false>))
                          : (unit ? reinterpret_cast<const void *>(&rope_append_kernel<1, true>)
                                  : reinterpret_cast<const void *>(&rope_append_kernel<1, false>));
    return launch_pdl(fn, dim3((unsigned)grid), kThreadsR, 0, stream, args);
}

}  // namespace nvfp4kv
