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
// Eight threads hold a row, 16 values each (one block of the format); the partner of a
// half-split pair comes by shuffle.  A thread takes up to kRows rows of one token, all
// loaded first, so that the token's table row, 128 bytes a thread, is read once for them.
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
    int chunks;                                      // thread groups a token
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

__device__ __forceinline__ float bf16_at(const uint32_t (&w)[8], int i) { return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }

__device__ __forceinline__ void unpack8(const uint4 &a, const uint4 &b, uint32_t (&w)[8]) {
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
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

// One row's block: x (this thread's 16 values), xp (the partner block's, half-split) and
// the weights -> 16 BF16 numbers.  c, s: the block's cosines and sines (adjacent pairs: 8
// of each, half-split: 16, the sines negated for the first half).  EXACT: see above.
template <bool EXACT>
__device__ __forceinline__ void turn_block(const RopeArgs &a, const uint32_t (&x)[8], const uint4 *weight, int blk, int pblk,
                                           unsigned group, int src, bool turned, const float (&c)[16], const float (&s)[16],
                                           uint32_t (&out)[8]) {
    uint32_t xp[8], w[8], wp[8];
    const bool half = !a.adjacent;
#pragma unroll
    for (int i = 0; i < 8; i++) xp[i] = x[i];
    if (half && a.rot) {
#pragma unroll
        for (int i = 0; i < 8; i++) xp[i] = __shfl_sync(group, x[i], src);
    }
    Pair r = {1.0f, 0.0f};
    if (weight) {
        unpack8(__ldg(weight + 2 * blk), __ldg(weight + 2 * blk + 1), w);
        unpack8(__ldg(weight + 2 * pblk), __ldg(weight + 2 * pblk + 1), wp);
        Pair q = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float v = bf16_at(x, i);
            if (EXACT) {                                    // (a BF16 number's square is exact)
                const Pair n = two_sum(q.hi, __fmul_rn(v, v));
                q = {n.hi, q.lo + n.lo};
            } else {
                q.hi = fmaf(v, v, q.hi);
            }
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
            const float h = __shfl_xor_sync(group, q.hi, d);
            if (EXACT) {
                const float l = __shfl_xor_sync(group, q.lo, d);
                const Pair n = two_sum(q.hi, h);
                q = {n.hi, (q.lo + l) + n.lo};
            } else {
                q.hi += h;
            }
        }
        if (EXACT) r = root(q, a.eps);
        else r.hi = rsqrtf(fmaf(q.hi, 0.0078125f, a.eps));
    }
    auto value = [&](int i) { return weight ? bf16_at(x, i) * bf16_at(w, i) : bf16_at(x, i); };      // exact: 16 bits
    auto partner = [&](int i) { return weight ? bf16_at(xp, i) * bf16_at(wp, i) : bf16_at(xp, i); };
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        float u[2] = {value(i), value(i + 1)}, p[2], cc[2], ss[2];
        if (half) {
#pragma unroll
            for (int e = 0; e < 2; e++) p[e] = partner(i + e), cc[e] = c[i + e], ss[e] = s[i + e];
        } else {
            p[0] = u[1], p[1] = u[0];
            cc[0] = cc[1] = c[i >> 1];
            ss[0] = -s[i >> 1], ss[1] = s[i >> 1];
        }
        uint32_t y[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
            if (EXACT) {
                Pair d = {u[e], 0.0f};
                if (turned) {
                    const float h = __fmul_rn(u[e], cc[e]), g = __fmul_rn(p[e], ss[e]);
                    const Pair z = two_sum(h, g);
                    d = {z.hi, z.lo + (__fmaf_rn(u[e], cc[e], -h) + __fmaf_rn(p[e], ss[e], -g))};
                }
                if (weight) {
                    const float h = __fmul_rn(d.hi, r.hi);
                    d = {h, __fmaf_rn(d.lo, r.hi, __fmaf_rn(d.hi, r.lo, __fmaf_rn(d.hi, r.hi, -h)))};
                }
                y[e] = bf16_of_pair(d.hi, d.lo);
            } else {
                float d = turned ? fmaf(u[e], cc[e], p[e] * ss[e]) : u[e];
                if (weight) d *= r.hi;
                y[e] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(d));
            }
        }
        out[i >> 1] = y[0] | (y[1] << 16);
    }
}

// Thread group g of eight (one row at a time) takes rows chunk + j * chunks of its token
// (rows: Hq of Q, then Hkv of K, then Hkv of V), j < kRows.
template <int kRows, bool kUnitScale>
__global__ void __launch_bounds__(kThreadsR) rope_append_kernel(RopeArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t id = (int64_t)blockIdx.x * (kThreadsR / 8) + (threadIdx.x >> 3);
    const int blk = threadIdx.x & 7, lane = threadIdx.x & 31;
    const unsigned group = 0xffu << (lane & 24);
    if (id >= a.num_tokens * a.chunks) return;               // (a whole group at a time)
    const int64_t t = id / a.chunks;
    const int chunk = (int)(id - t * a.chunks), rows = a.Hq + 2 * a.Hkv;
    uint4 x0[kRows], x1[kRows];
#pragma unroll
    for (int j = 0; j < kRows; j++) {
        const int row = chunk + j * a.chunks;
        if (row >= rows) continue;
        const uint4 *src = row < a.Hq ? a.q + t * a.q_stride16 + row * 16
                           : row < a.Hq + a.Hkv ? a.k + t * a.kv_stride16 + (row - a.Hq) * 16
                                                : a.v + t * a.kv_stride16 + (row - a.Hq - a.Hkv) * 16;
        x0[j] = __ldg(src + 2 * blk);
        x1[j] = __ldg(src + 2 * blk + 1);
    }
    const int64_t slot = __ldg(a.slots + t);
    // ---- the block's pairs, and their row of the table (a float4 of pairs lies in one section)
    const int half16 = a.rot >> 5;                           // blocks of half the rotated values
    const bool turned = blk < (a.rot >> 4);
    const bool second = !a.adjacent && blk >= half16;
    const int pblk = !turned || a.adjacent ? blk : second ? blk - half16 : blk + half16;
    float c[16], s[16];
    bool ok = true;
    if (turned) {
        const int first = a.adjacent ? 8 * blk : 16 * (second ? blk - half16 : blk), n4 = a.adjacent ? 2 : 4;
        const float4 *at[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (i >= n4) continue;
            const int pair = first + 4 * i, axis = pair < a.sec1 ? 0 : pair < a.sec2 ? 1 : 2;
            const int32_t pos = __ldg(a.positions + axis * a.num_tokens + t);
            const bool in = pos >= 0 && pos < a.num_positions;
            ok = ok && in;
            at[i] = reinterpret_cast<const float4 *>(a.table + (in ? (int64_t)pos * a.rot : 0) + pair);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (i >= n4) continue;
            const float4 x = __ldg(at[i]), y = __ldg(at[i] + (a.rot >> 3));
            const float f = !a.adjacent && !second ? -1.0f : 1.0f;
            c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
            s[4 * i] = f * y.x, s[4 * i + 1] = f * y.y, s[4 * i + 2] = f * y.z, s[4 * i + 3] = f * y.w;
        }
    }
    ok = __all_sync(group, ok);
    if (!ok && blk == 0 && chunk == 0) flag_error(a.err, kErrPosition);
    if (slot >= a.num_slots && blk == 0 && chunk == 0) flag_error(a.err, kErrSlot);
    const bool write = slot >= 0 && slot < a.num_slots;
    if (!ok) return;
    const int64_t page = write ? slot >> a.log2P : 0;
    const int in_page = (int)(slot & (a.P - 1));
    const int src = (lane & 24) + pblk;
    const uint64_t policy = l2_policy_evict_last();          // of scale bytes, as in the plain append
#pragma unroll
    for (int j = 0; j < kRows; j++) {
        const int row = chunk + j * a.chunks;
        if (row >= rows) continue;
        uint32_t x[8], y[8];
        unpack8(x0[j], x1[j], x);
        if (row < a.Hq) {
            turn_block<false>(a, x, a.wq, blk, pblk, group, src, turned, c, s, y);
            uint4 *dst = a.q_out + t * a.out_stride16 + row * 16 + 2 * blk;
            dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
            dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
        } else if (write) {
            const int which = row >= a.Hq + a.Hkv;
            uint4 y0 = x0[j], y1 = x1[j];
            if (!which) {
                turn_block<true>(a, x, a.wk, blk, pblk, group, src, turned, c, s, y);
                y0 = make_uint4(y[0], y[1], y[2], y[3]);
                y1 = make_uint4(y[4], y[5], y[6], y[7]);
            }
            const int h = row - a.Hq - which * a.Hkv;
            store_block_values<kUnitScale, true>(a.pool + (page * a.Hkv + h) * a.slab, a.dtype, in_page, which, blk, y0, y1,
                                                 which ? a.gv : a.gk, policy);
        }
    }
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
    // One row a thread while that does not fill the GPU (152 SMs of 2,048 threads), four beyond.
    const int rows = a.Hq + 2 * a.Hkv;
    const bool many = num_tokens * rows * 8 > 152 * 2048;
    a.chunks = many ? (rows + 3) / 4 : rows;
    const int64_t grid = ceil_div64(num_tokens * a.chunks, kThreadsR / 8);
    const bool unit = c.k_global_scale == 1.0f && c.v_global_scale == 1.0f;
    void *args[] = {&a};
    const void *fn = many ? (unit ? reinterpret_cast<const void *>(&rope_append_kernel<4, true>)
                                  : reinterpret_cast<const void *>(&rope_append_kernel<4, false>))
                          : (unit ? reinterpret_cast<const void *>(&rope_append_kernel<1, true>)
                                  : reinterpret_cast<const void *>(&rope_append_kernel<1, false>));
    return launch_pdl(fn, dim3((unsigned)grid), kThreadsR, 0, stream, args);
}

}  // namespace nvfp4kv
