// latent_decode.cu -- absorbed latent attention of one query a sequence over the paged latent cache.
//
//   s[h][t] = q_latent[h] . c_t + q_rope[h] . r_t,   out[h] = sum_t softmax_t(sm_scale s[h][t]) c_t
// All heads share the token's 512-value latent c_t (NVFP4) and 64-value rotary
// part r_t (BF16), so a token costs 416 bytes and 2 * 1,088 flops a head: with 16
// heads the cache's bytes bound it, with 128 the tensor cores.
//
// Tokens sit on the tensor core's M dimension in both products, heads on N:
//   S^T (128 tokens x N heads)  = C Q^T    36 steps of M 128 x N x K 16
//   O^T (512 dims  x N heads)  += C^T P^T  4 row blocks x 8 steps
// so 16 heads fill N = 16 with no padding (heads on M would be padded to 128 rows),
// and one FP16 copy of the tile in shared memory, [8 column blocks][128 tokens][64
// dims] with the 128-byte swizzle, is the K-major A operand of the first product
// and the MN-major A operand of the second.  e2m1 x e4m3 is an exact FP16 value;
// the tensor scale is folded into q (FP16 after a power-of-two pre-scale a head,
// exact for g = 1 above 2^-29 of its largest value) and into the output; the
// rotary steps are BF16 into the same accumulator.
//
// One CTA per SM.  Eight warps do everything but issue the products:
//   * warp w holds the raw bytes of the tile's w-th 16-token group in registers
//     (13 16-byte loads a lane, requested a whole tile ahead, straight from the
//     page) and expands them into the tile, two column blocks at a time: pair i as
//     soon as O += of row block i of the previous tile has read it;
//   * then they run the softmax of the 128 x N scores, one token a thread, the two
//     warpgroups taking half the heads each: base 2 with a lazily moved maximum per
//     head (a vote over the warpgroup; O^T is rescaled only when a score exceeds the
//     maximum by 2^8), P = 2^(s - m + 7) in FP16 (the offset uses FP16's upper
//     range: weights down to 2^-21 of the largest keep full precision) over the
//     rotary tile, whose product is done; the row sums of the rounded P stay in
//     registers, one (token, head) each, until the sequence ends.
// One thread of warp 8 issues S^T as the pairs arrive and O^T per row block.
//
// Split: the batch's 128-token tiles form one flat range, cut equally over the
// CTAs of a head tile (64 heads).  A sequence that lies in one CTA is normalised
// and written there; others leave (m, l, O) partials that a second kernel joins.
// Every wait is bounded.
#include <mutex>

#include "common.cuh"
#include "flat_plan.cuh"
#include "kernels.h"
#include "latent.cuh"
#include "quantize.cuh"
#include "tcgen05.cuh"

namespace nvfp4kv {

namespace {

constexpr int kWorkers = 256;                 // expanding and softmax threads
constexpr int kLThreads = kWorkers + 128;     // + the MMA warp's warpgroup (its other warps only meet the last barrier)
// Launched with 168 registers a thread; the two working warpgroups then take 216
// and the third gives back down to 72: 2 x 128 x 216 + 128 x 72 = 384 x 168.
constexpr int kWorkRegs = 216, kMmaRegs = 72;
static_assert(2 * 128 * kWorkRegs + 128 * kMmaRegs <= kLThreads * 168, "register split must fit the launch");
constexpr int kTile = 128;                    // tokens per tile
constexpr int kColBlock = kTile * 128;        // bytes of one column block (64 dims) of the tile
constexpr int kTileBytes = 8 * kColBlock;
constexpr uint32_t kWaitLimitL = 1u << 22;
constexpr float kNegInfL = -__builtin_huge_valf();
constexpr float kRescaleL = 8.0f;
constexpr float kPOffset = 7.0f;              // P = 2^(s - m + 7): at most 2^15
constexpr int kNumBarsL = 12;                 // kv_full[5] s_done p_full pv_done[4] drain

template <int N>
struct LSmem {
    static constexpr int kQBlock = N * 128;               // one column block of Q, [N][64]
    static constexpr int kQ = 0;                          // 8 FP16 blocks + the BF16 rotary block
    static constexpr int kKV = 9 * kQBlock;
    static constexpr int kRope = kKV + kTileBytes;        // BF16 [128][64]; P over it: FP16 [128 tokens][N]
    static constexpr int kBar = kRope + kColBlock;
    static constexpr int kMisc = kBar + kNumBarsL * 8;    // tmem base, abort
    static constexpr int kM = kMisc + 16;                 // float m[N], fac[N], alpha[N]
    static constexpr int kWarpMax = kM + 3 * N * 4;       // float [2][4][N / 2]
    static constexpr int kWarpSum = kWarpMax + 4 * N * 4; // float [2][4][N / 2]
    static constexpr int kBytes = kWarpSum + 4 * N * 4;
    static constexpr uint32_t kCols = N == 64 ? 512 : N == 32 ? 256 : 128;   // O at 0 .. 4N, S at 4N .. 5N
    static_assert(kKV % 1024 == 0 && kRope % 1024 == 0, "operand tiles need 1024-byte alignment");
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static_assert(sizeof(FlatScratch<kLThreads>) <= kTileBytes, "the plan's scratch lies in the tile");
};

struct LatentArgs {
    const uint8_t *pool;
    int64_t num_pages;
    int P, log2P, B, H, max_pages;
    const int32_t *block_table, *seq_lens;
    int64_t cap;
    const uint16_t *ql, *qr;
    float score_log2;       // sm_scale * log2(e)
    float g;
    __nv_bfloat16 *out;
    float2 *part_ml;        // [splits + B][H]
    float *part_acc;        // [splits + B][H][512]
    int splits;
    unsigned *err;
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const volatile int *abort_flag) {
    for (uint32_t n = 0; n < kWaitLimitL; n++) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
    }
    return false;
}

// The tiles of a CTA's range in order.
struct TileIter {
    int b, t, nt, n;
    int64_t left;   // tiles of the range from this one on
};

__device__ __forceinline__ void set_seq(const LatentArgs &a, TileIter &it) {
    it.n = clamp_rows(__ldg(a.seq_lens + it.b), a.cap);
    it.nt = (it.n + kTile - 1) / kTile;
}

__device__ __forceinline__ void next_tile(const LatentArgs &a, TileIter &it) {
    it.left--;
    if (++it.t < it.nt || it.left <= 0) return;
    it.t = 0;
    do {            // left > 0: a later sequence has tiles
        it.b++;
        set_seq(a, it);
    } while (it.nt == 0);
}

// s0 += low FP16 of w, s1 += high FP16 of w
__device__ __forceinline__ void add_f16x2(float &s0, float &s1, uint32_t w) {
    const unsigned short one = 0x3c00;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2;\n"
        "fma.rn.f32.f16 %0, lo, %3, %0; fma.rn.f32.f16 %1, hi, %3, %1; }"
        : "+f"(s0), "+f"(s1)
        : "r"(w), "h"(one));
}

// Barriers 1 and 2: the warpgroups; 3: both.
__device__ __forceinline__ void group_sync(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); }
__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

__device__ __forceinline__ bool group_any(int wg, bool p) {
    uint32_t r;
    asm volatile("{ .reg .pred a, b; setp.ne.u32 a, %2, 0; bar.red.or.pred b, %1, 128, a; selp.u32 %0, 1, 0, b; }"
                 : "=r"(r)
                 : "r"(1 + wg), "r"((uint32_t)p)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// v[c] (c < CW <= 32) summed over the warp's lanes: lane c returns column c's sum (lanes >= CW: a copy of c % CW's)
template <int CW>
__device__ __forceinline__ float column_sums(float (&v)[CW], int lane) {
#pragma unroll
    for (int w = CW / 2; w; w >>= 1) {   // halve the columns, each half of the lanes keeping one half of them
        const bool up = lane & w;
#pragma unroll
        for (int c = 0; c < CW / 2; c++) {
            if (c >= w) break;
            const float send = up ? v[c] : v[c + w];
            const float keep = up ? v[c + w] : v[c];
            v[c] = keep + __shfl_xor_sync(0xffffffffu, send, w);
        }
    }
    float s = v[0];
#pragma unroll
    for (int w = CW; w < 32; w <<= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    return s;
}

template <int N>
__global__ void __launch_bounds__(kLThreads, 1) latent_decode_kernel(LatentArgs a) {
    using L = LSmem<N>;
    constexpr int CW = N / 2;                     // heads per warpgroup
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBar);
    uint64_t *kv_full = bars, *s_done = bars + 5, *p_full = bars + 6, *pv_done = bars + 7, *drain = bars + 11;
    uint32_t &tmem_base = *reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    float *s_m = reinterpret_cast<float *>(smem + L::kM), *s_fac = s_m + N, *s_alpha = s_fac + N;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h0 = blockIdx.y * N;
    pdl_wait();               // everything read or written may belong to earlier work of the stream
    pdl_launch_dependents();

    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = tid; b < a.B; b += kLThreads) {
            const int32_t n = a.seq_lens[b];
            if (n < 0 || (int64_t)n > a.cap) flag_error(a.err, kErrSeqLen);
        }
    int b0;
    int64_t first, u0 = 0;
    const int64_t total = flat_locate<kLThreads>(
        *reinterpret_cast<FlatScratch<kLThreads> *>(smem + L::kKV), a.B,
        [&](int b) { return (int64_t)((clamp_rows(__ldg(a.seq_lens + b), a.cap) + kTile - 1) / kTile); },
        [&](int64_t t) { return u0 = flat_begin(blockIdx.x, t, a.splits); }, b0, first);
    const int64_t u1 = flat_begin((int64_t)blockIdx.x + 1, total, a.splits);
    if (u0 >= u1) return;
    TileIter it;
    it.b = b0;
    it.t = (int)(u0 - first);
    it.left = u1 - u0;
    set_seq(a, it);

    if (warp == 8) tc_alloc(&tmem_base, L::kCols);
    if (tid == 0) {
        for (int i = 0; i < kNumBarsL; i++) mbar_init(&bars[i], i < 5 || i == 6 ? kWorkers / 32 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base, sbase = smem_u32(smem);
    constexpr uint32_t kColS = 4 * N;

    if (warp >= 8) {
        // ---------------- the MMA thread
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
        // The whole warp runs the loop and one elected lane issues, so that the compiler
        // sees the descriptors as uniform values: a product issued under a divergent
        // branch cost 70 to 110 clocks, more than the products themselves (38 at N = 16,
        // 47 at N = 64).
        if (warp == 8) {
            bool ok = true;
            constexpr uint32_t idesc_s = idesc_f16_f32(128, N, false), idesc_r = idesc_bf16_f32(128, N, false);
            constexpr uint32_t idesc_o = idesc_a_mn_major(idesc_f16_f32(128, N, true));
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const bool leader = elect_one();
            // operand descriptors; a step adds its byte offset / 16 to the address field
            const uint64_t dC = smem_desc_sw128(sbase + L::kKV, 16, 1024), dQ = smem_desc_sw128(sbase + L::kQ, 16, 1024);
            const uint64_t dR = smem_desc_sw128(sbase + L::kRope, 16, 1024);   // rotary tile, and P over it
            const uint64_t dV = smem_desc_sw128(sbase + L::kKV, kColBlock, 1024);
            bool fresh = true;   // the tile is the range's first of its sequence
            for (uint32_t j = 0; it.left > 0; j++) {
#pragma unroll 1
                for (uint32_t i = 0; i < 4; i++) {
                    ok = ok && wait_bar(&kv_full[i], j & 1, abort_flag);
                    tc_fence_after();
                    if (leader) {
                        const uint64_t dCi = dC + i * (2 * kColBlock / 16), dQi = dQ + i * (2 * L::kQBlock / 16);
#pragma unroll
                        for (int kk = 0; kk < 8; kk++) {
                            const uint32_t half = kk >> 2, sub = (uint32_t)(kk & 3) * 2;
                            tc_mma_bf16(tm + kColS, dCi + (half * (kColBlock / 16) + sub), dQi + (half * (L::kQBlock / 16) + sub),
                                        idesc_s, i > 0 || kk > 0);
                        }
                    }
                }
                ok = ok && wait_bar(&kv_full[4], j & 1, abort_flag);
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 4; kk++)
                        tc_mma_bf16(tm + kColS, dR + kk * 2, dQ + (8 * L::kQBlock / 16 + kk * 2), idesc_r, 1u);
                    tc_commit(s_done);
                }
                ok = ok && wait_bar(p_full, j & 1, abort_flag);
                tc_fence_after();
                if (!__all_sync(0xffffffffu, ok)) break;
                if (leader) {
                    const uint32_t acc = fresh ? 0u : 1u;
#pragma unroll 1
                    for (uint32_t mb = 0; mb < 4; mb++) {
                        const uint64_t dVm = dV + mb * (2 * kColBlock / 16);
#pragma unroll
                        for (int kk = 0; kk < 8; kk++)   // 16 tokens: 2,048 bytes of a column block, and of P
                            tc_mma_bf16(tm + mb * N, dVm + kk * 128, dR + kk * 128, idesc_o,
                                        kk > 0 ? 1u : acc);
                        tc_commit(&pv_done[mb]);
                    }
                }
                const int b = it.b;
                next_tile(a, it);
                fresh = it.b != b;
            }
            if (!__all_sync(0xffffffffu, ok) && leader) {
                if (!*abort_flag) flag_error(a.err, kErrTimeout);
                *abort_flag = 1;
                tc_commit(drain);   // no product may still read the CTA's memory when it ends
                mbar_wait_bounded(drain, 0, kWaitLimitL, nullptr);
            }
        }
        __syncwarp();
    } else {
        // ---------------- expanding and softmax warps
        // A wait that gave up sets the abort flag, which ends every other wait; the
        // warps then still run through their tiles (on meaningless values), so that
        // no barrier is left short of a warp.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWorkRegs));
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!wait_bar(bar, parity, abort_flag) && !*abort_flag) {
                *abort_flag = 1;
                flag_error(a.err, kErrTimeout);
            }
        };
        const int wg = warp >> 2, row = 32 * (warp & 3) + lane;   // softmax: this thread's token (TMEM lane)
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int er = lane >> 1, hb = lane & 1;                  // expanding: row of the group, half of a column block
        uint4 code[8], scl, rope[4];
        auto page_of = [&](const TileIter &x) -> int32_t {        // page of this warp's group (-1: none)
            const int t = x.t * kTile + 16 * warp;
            if (x.left <= 0 || t >= x.n) return -1;
            return __ldg(a.block_table + (int64_t)x.b * a.max_pages + (t >> a.log2P));
        };
        auto load_tile = [&](const TileIter &x, int32_t page) {
            const int t = x.t * kTile + 16 * warp;
            const bool there = x.left > 0 && t < x.n;
            const bool good = there && page >= 0 && page < a.num_pages;
            if (there && !good && lane == 0) flag_error(a.err, kErrPage);
            const uint8_t *grp = a.pool + (int64_t)(good ? page : 0) * ((int64_t)kLatentRow * a.P) +
                                 (int64_t)((t & (a.P - 1)) >> 4) * kLatentGroup;
            const bool rok = good && t + er < x.n;
#pragma unroll
            for (int cb = 0; cb < 8; cb++)
                code[cb] = rok ? __ldg(reinterpret_cast<const uint4 *>(grp + cb * 512 + lane * 16)) : make_uint4(0, 0, 0, 0);
            scl = rok ? __ldg(reinterpret_cast<const uint4 *>(grp + kLatentScales + lane * 16)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int x4 = 0; x4 < 4; x4++)
                rope[x4] = good && t + 4 * x4 + (lane >> 3) < x.n
                               ? __ldg(reinterpret_cast<const uint4 *>(grp + kLatentRope + x4 * 512 + lane * 16))
                               : make_uint4(0, 0, 0, 0);
        };
        TileIter nx = it;                       // the tile whose bytes are requested next
        load_tile(nx, page_of(nx));
        next_tile(a, nx);
        int32_t npage = page_of(nx);            // its page, requested a tile earlier still
        bool fresh = true;
        int t_begin = it.t;                     // first tile of the current sequence in this range
        float l[CW];
        for (uint32_t j = 0; it.left > 0; j++) {
            if (fresh) {
                // ---- Q of the sequence: one warp per head, FP16 latent blocks and the BF16 rotary block
                // (S of the previous sequence is done: its scores were read)
                for (int hh = warp; hh < N; hh += 8) {
                    const int h = h0 + hh;
                    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
                    uint32_t xr = 0;
                    if (h < a.H) {
                        const int64_t at = (int64_t)it.b * a.H + h;
                        const uint4 *src = reinterpret_cast<const uint4 *>(a.ql + at * kLatentDim) + lane * 2;
                        x0 = __ldg(src);
                        x1 = __ldg(src + 1);
                        xr = __ldg(reinterpret_cast<const uint32_t *>(a.qr + at * kRopeDim) + lane);
                    }
                    const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                    uint32_t ml = 0, mr = xr & 0x7fff7fffu;
#pragma unroll
                    for (int e = 0; e < 8; e++) ml = max_u16x2(ml, w[e] & 0x7fff7fffu);
                    ml = __reduce_max_sync(0xffffffffu, max(ml >> 16, ml & 0xffffu));
                    mr = __reduce_max_sync(0xffffffffu, max(mr >> 16, mr & 0xffffu));
                    // 2^kq puts the largest |q g| into [2^14, 2^15), the rotary part below 2^127
                    const uint32_t top = __float_as_uint(__uint_as_float(ml << 16) * a.g);
                    int kq = top ? 14 - ((int)(top >> 23) - 127) : 0;
                    kq = min(min(126, max(-126, kq)), 126 - ((int)(mr >> 7) - 127));
                    kq = max(-126, kq);
                    const float sc = __uint_as_float((uint32_t)(kq + 127) << 23);
                    uint32_t f[8];
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        f[e] = f32x2_to_f16x2(bf16_hi(w[e]) * a.g * sc, bf16_lo(w[e]) * a.g * sc);
                    uint8_t *q = smem + L::kQ + (lane >> 2) * L::kQBlock;      // lane: dims 16 lane .. 16 lane + 15
                    *reinterpret_cast<uint4 *>(q + sw128_off(hh, (lane & 3) * 2)) = make_uint4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<uint4 *>(q + sw128_off(hh, (lane & 3) * 2 + 1)) = make_uint4(f[4], f[5], f[6], f[7]);
                    *reinterpret_cast<uint32_t *>(smem + L::kQ + 8 * L::kQBlock + sw128_off(hh, lane >> 2) + (lane & 3) * 4) =
                        f32x2_to_bf16x2(bf16_hi(xr) * sc, bf16_lo(xr) * sc);
                    if (lane == 0) {
                        s_fac[hh] = a.score_log2 * __uint_as_float((uint32_t)(127 - kq) << 23);
                        s_m[hh] = kNegInfL;
                    }
                }
#pragma unroll
                for (int c = 0; c < CW; c++) l[c] = 0.f;
                workers_sync();   // s_fac and s_m are written for all heads
            }
            // ---- expand the tile, a pair of column blocks at a time
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (j > 0) wait(&pv_done[i], (j - 1) & 1);
                const uint4 wv[2] = {code[2 * i], code[2 * i + 1]};
                const uint32_t s4 = i == 0 ? scl.x : i == 1 ? scl.y : i == 2 ? scl.z : scl.w;
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    const uint32_t s2 = e4m3x2_to_f16x2((s4 >> (16 * c)) & 0xffffu);
                    const uint32_t lo = __byte_perm(s2, s2, 0x1010), hi = __byte_perm(s2, s2, 0x3232);
                    uint32_t f[16];
                    e2m1x8_to_f16x2x4(wv[c].x, f[0], f[1], f[2], f[3]);
                    e2m1x8_to_f16x2x4(wv[c].y, f[4], f[5], f[6], f[7]);
                    e2m1x8_to_f16x2x4(wv[c].z, f[8], f[9], f[10], f[11]);
                    e2m1x8_to_f16x2x4(wv[c].w, f[12], f[13], f[14], f[15]);
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        f[e] = hmul2(f[e], lo);
                        f[8 + e] = hmul2(f[8 + e], hi);
                    }
                    uint8_t *blk = smem + L::kKV + (2 * i + c) * kColBlock;
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        *reinterpret_cast<uint4 *>(blk + sw128_off(16 * warp + er, 4 * hb + k)) =
                            make_uint4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&kv_full[i]);
            }
            // the rotary tile, over the previous tile's P (row block 3, the last to read it, is done)
#pragma unroll
            for (int x4 = 0; x4 < 4; x4++)
                *reinterpret_cast<uint4 *>(smem + L::kRope + warp * 2048 + x4 * 512 + lane * 16) = rope[x4];
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&kv_full[4]);
            // ---- request the next tile's bytes, and the page after that
            load_tile(nx, npage);
            next_tile(a, nx);
            npage = page_of(nx);

            // ---- softmax of this thread's token
            wait(s_done, j & 1);
            __syncwarp();
            tc_fence_after();
            const bool seen = it.t * kTile + row < it.n;
            uint32_t sr[CW];
            tc_ld(tmem + lanes + kColS + wg * CW, sr);
            tc_wait_ld();
            float sc[CW];
            bool need = false;
#pragma unroll
            for (int c = 0; c < CW; c++) {
                sc[c] = seen ? __uint_as_float(sr[c]) * s_fac[wg * CW + c] : kNegInfL;
                need |= sc[c] > s_m[wg * CW + c] + kRescaleL;
            }
            if (group_any(wg, need)) {
                float *wmax = reinterpret_cast<float *>(smem + L::kWarpMax) + wg * 4 * CW;
                int mine = 0;
#pragma unroll
                for (int c = 0; c < CW; c++) {
                    const int mx = __reduce_max_sync(0xffffffffu, ordered(sc[c]));
                    if (lane == c) mine = mx;
                }
                if (lane < CW) wmax[(warp & 3) * CW + lane] = unordered(mine);
                group_sync(wg);
                if ((warp & 3) == 0 && lane < CW) {
                    const float mx = fmaxf(fmaxf(wmax[lane], wmax[CW + lane]), fmaxf(wmax[2 * CW + lane], wmax[3 * CW + lane]));
                    const float mo = s_m[wg * CW + lane], mn = fmaxf(mo, mx);
                    s_alpha[wg * CW + lane] = mo == kNegInfL ? 0.f : ex2(mo - mn);
                    s_m[wg * CW + lane] = mn;
                }
                group_sync(wg);
#pragma unroll
                for (int c = 0; c < CW; c++) l[c] *= s_alpha[wg * CW + c];
                if (!fresh) {   // O^T holds earlier tiles, complete: rescale this warp's lanes of the warpgroup's heads
#pragma unroll 1
                    for (int mb = 0; mb < 4; mb++) {
                        uint32_t ov[CW];
                        tc_ld(tmem + lanes + mb * N + wg * CW, ov);
                        tc_wait_ld();
#pragma unroll
                        for (int c = 0; c < CW; c++)
                            ov[c] = __float_as_uint(__uint_as_float(ov[c]) * s_alpha[wg * CW + c]);
                        tc_st(tmem + lanes + mb * N + wg * CW, ov);
                    }
                    tc_wait_st();
                }
            }
#pragma unroll
            for (int k = 0; k < CW / 8; k++) {
                uint32_t pw[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int c = 8 * k + 2 * e;
                    const float m0 = s_m[wg * CW + c], m1 = s_m[wg * CW + c + 1];
                    pw[e] = f32x2_to_f16x2(ex2(sc[c + 1] - (m1 == kNegInfL ? 0.f : m1 - kPOffset)),
                                           ex2(sc[c] - (m0 == kNegInfL ? 0.f : m0 - kPOffset)));
                    add_f16x2(l[c], l[c + 1], pw[e]);
                }
                *reinterpret_cast<uint4 *>(smem + L::kRope + sw128_off(row, wg * (CW / 8) + k)) =
                    make_uint4(pw[0], pw[1], pw[2], pw[3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);

            // ---- the sequence's last tile of this range: normalise, or leave the partial
            const TileIter cur = it;
            next_tile(a, it);
            fresh = it.left <= 0 || it.b != cur.b;
            if (!fresh) continue;
            for (int i = 0; i < 4; i++) wait(&pv_done[i], j & 1);
            __syncwarp();
            tc_fence_after();
            {
                float *wsum = reinterpret_cast<float *>(smem + L::kWarpSum) + wg * 4 * CW;
                const float s = column_sums<CW>(l, lane);
                if (lane < CW) wsum[(warp & 3) * CW + lane] = s;
                group_sync(wg);
                const bool whole = t_begin == 0 && cur.t == cur.nt - 1;
                const int64_t slot = (int64_t)blockIdx.x + cur.b;
                if (!whole && (warp & 3) == 0 && lane < CW && h0 + wg * CW + lane < a.H) {
                    const float m = s_m[wg * CW + lane];
                    a.part_ml[slot * a.H + h0 + wg * CW + lane] = make_float2(
                        m == kNegInfL ? m : m - kPOffset,
                        (wsum[lane] + wsum[CW + lane]) + (wsum[2 * CW + lane] + wsum[3 * CW + lane]));
                }
#pragma unroll 1
                for (int mb = 0; mb < 4; mb++) {
                    uint32_t ov[CW];
                    tc_ld(tmem + lanes + mb * N + wg * CW, ov);
                    tc_wait_ld();
                    const int d = mb * 128 + row;
#pragma unroll
                    for (int c = 0; c < CW; c++) {
                        const int h = h0 + wg * CW + c;
                        if (h >= a.H) continue;
                        const float o = __uint_as_float(ov[c]);
                        if (whole) {
                            const float ls = (wsum[c] + wsum[CW + c]) + (wsum[2 * CW + c] + wsum[3 * CW + c]);
                            a.out[((int64_t)cur.b * a.H + h) * kLatentDim + d] = __float2bfloat16_rn(o * (a.g / ls));
                        } else {
                            a.part_acc[(slot * a.H + h) * kLatentDim + d] = o;
                        }
                    }
                }
                tc_fence_before();
                workers_sync();   // wsum and s_m are read: the next sequence may write them
            }
            t_begin = it.t;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tc_dealloc(tmem, L::kCols);
}

// Joins the partials of the sequences that several CTAs covered (and zeroes those
// of length 0): one CTA per (sequence, head), thread t owns dims 4t .. 4t + 3.
constexpr int kJoinThreads = 128;

__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(LatentArgs a) {
    __shared__ int64_t s_sum[2][kJoinThreads / 32];
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    auto tiles = [&](int x) { return (int64_t)((clamp_rows(__ldg(a.seq_lens + x), a.cap) + kTile - 1) / kTile); };
    int64_t before = 0, all = 0;
    for (int x = tid; x < a.B; x += kJoinThreads) {
        const int64_t t = tiles(x);
        all += t;
        if (x < b) before += t;
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, x);
        before += __shfl_xor_sync(0xffffffffu, before, x);
    }
    if ((tid & 31) == 0) {
        s_sum[0][tid >> 5] = all;
        s_sum[1][tid >> 5] = before;
    }
    __syncthreads();
    all = before = 0;
    for (int w = 0; w < kJoinThreads / 32; w++) {
        all += s_sum[0][w];
        before += s_sum[1][w];
    }
    const int64_t nt = tiles(b);
    uint2 *dst = reinterpret_cast<uint2 *>(a.out + ((int64_t)b * a.H + h) * kLatentDim) + tid;
    if (nt == 0) {
        *dst = make_uint2(0, 0);
        return;
    }
    const int64_t c0 = flat_piece(before, all, a.splits), c1 = flat_piece(before + nt - 1, all, a.splits);
    if (c0 == c1) return;   // written by its CTA
    float m = kNegInfL, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t c = c0; c <= c1; c += 4) {
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            ml[k] = make_float2(kNegInfL, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + k <= c1) {   // every CTA between c0 and c1 holds tiles of the sequence (none is empty between two that do)
                const int64_t cc = c + k;
                if (flat_begin(cc, all, a.splits) < flat_begin(cc + 1, all, a.splits)) {
                    const int64_t at = (cc + b) * a.H + h;
                    ml[k] = __ldcg(a.part_ml + at);
                    v[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_acc + at * kLatentDim) + tid);
                }
            }
        }
        float mx = m;
#pragma unroll
        for (int k = 0; k < 4; k++) mx = fmaxf(mx, ml[k].x);
        const float f0 = m == kNegInfL ? 0.f : ex2(m - mx);
        l *= f0;
        acc.x *= f0;
        acc.y *= f0;
        acc.z *= f0;
        acc.w *= f0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float f = ml[k].x == kNegInfL ? 0.f : ex2(ml[k].x - mx);
            l += f * ml[k].y;
            acc.x += f * v[k].x;
            acc.y += f * v[k].y;
            acc.z += f * v[k].z;
            acc.w += f * v[k].w;
        }
        m = mx;
    }
    const float inv = a.g / l;
    *dst = make_uint2(f32x2_to_bf16x2(acc.y * inv, acc.x * inv), f32x2_to_bf16x2(acc.w * inv, acc.z * inv));
}

int tile_heads(int H) { return H <= 16 ? 16 : H <= 32 ? 32 : 64; }

const void *decode_fn(int n, int *smem) {
    if (n == 16) {
        *smem = LSmem<16>::kBytes;
        return reinterpret_cast<const void *>(&latent_decode_kernel<16>);
    }
    if (n == 32) {
        *smem = LSmem<32>::kBytes;
        return reinterpret_cast<const void *>(&latent_decode_kernel<32>);
    }
    *smem = LSmem<64>::kBytes;
    return reinterpret_cast<const void *>(&latent_decode_kernel<64>);
}

constexpr int kMaxDevicesL = 64;
std::mutex g_mu_l;
bool g_attr_l[kMaxDevicesL][3];
int g_sms_l[kMaxDevicesL];

size_t align256l(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

int latent_decode_auto_splits(int num_heads, cudaError_t *status) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevicesL)) e = cudaErrorInvalidDevice;
    if (e == cudaSuccess) {
        std::lock_guard<std::mutex> lock(g_mu_l);
        if (!g_sms_l[dev]) e = cudaDeviceGetAttribute(&g_sms_l[dev], cudaDevAttrMultiProcessorCount, dev);
        sms = g_sms_l[dev];
    }
    if (status) *status = e;
    if (e != cudaSuccess) return 0;
    const int n = tile_heads(num_heads), tiles = (num_heads + n - 1) / n;
    return sms / tiles > 0 ? sms / tiles : 1;
}

// Workspace: (m, l) partials | their O, one per (CTA of a head tile, sequence) that can meet
size_t latent_decode_workspace_bytes(int batch, int num_heads, int splits) {
    const size_t slots = (size_t)splits + (size_t)batch;
    return align256l(slots * num_heads * sizeof(float2)) + slots * num_heads * kLatentDim * sizeof(float);
}

cudaError_t launch_latent_decode(const nvfp4kv_latent_cache &c, const void *q_latent, const void *q_rope, int batch,
                                 int num_heads, const int32_t *block_table, int max_pages, const int32_t *seq_lens,
                                 float sm_scale, void *out, void *workspace, int splits, unsigned *err,
                                 cudaStream_t stream) {
    const int n = tile_heads(num_heads), tiles = (num_heads + n - 1) / n;
    int dev = 0, smem = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevicesL) return cudaErrorInvalidDevice;
    const void *fn = decode_fn(n, &smem);
    {
        std::lock_guard<std::mutex> lock(g_mu_l);
        bool &set = g_attr_l[dev][n == 16 ? 0 : n == 32 ? 1 : 2];
        if (!set) {
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            set = true;
        }
    }
    LatentArgs a;
    a.pool = static_cast<const uint8_t *>(c.pool);
    a.num_pages = c.num_pages;
    a.P = c.page_size;
    a.log2P = __builtin_ctz((unsigned)c.page_size);
    a.B = batch;
    a.H = num_heads;
    a.max_pages = max_pages;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.cap = (int64_t)max_pages * c.page_size;
    a.ql = static_cast<const uint16_t *>(q_latent);
    a.qr = static_cast<const uint16_t *>(q_rope);
    a.score_log2 = (float)((double)sm_scale * 1.4426950408889634);
    a.g = c.global_scale;
    a.out = static_cast<__nv_bfloat16 *>(out);
    const size_t slots = (size_t)splits + (size_t)batch;
    a.part_ml = static_cast<float2 *>(workspace);
    a.part_acc = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + align256l(slots * num_heads * sizeof(float2)));
    a.splits = splits;
    a.err = err;
    void *args[] = {&a};
    e = launch_pdl(fn, dim3((unsigned)splits, (unsigned)tiles), kLThreads, (size_t)smem, stream, args);
    if (e != cudaSuccess) return e;
    return launch_pdl(reinterpret_cast<const void *>(&latent_join_kernel), dim3((unsigned)num_heads, (unsigned)batch),
                      kJoinThreads, 0, stream, args);
}

}  // namespace nvfp4kv
