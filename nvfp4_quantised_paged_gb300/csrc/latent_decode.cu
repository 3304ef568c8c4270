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
// rotary steps are BF16, by the same pre-scale, into the same accumulator.
//
// One CTA per SM.  Sixteen warps do everything but issue the products:
//   * expanding: two warps per 16-token group, taking every other column block; lane (r,
//     q) holds the raw bytes of block q (16 dims) of rows r and r + 8, loaded straight from
//     the page in contiguous pieces, each requested again for the next tile as soon as it
//     is used.  A block goes to the tile in shared memory, as soon as the previous tile's
//     O^T row block that reads it is done, and to TMEM as the A operand of S^T (all
//     column blocks up to 32 heads, the last four with 64; the rotary part to TMEM alone): an A
//     operand in shared memory costs a product 4 KB of reads, at least 38 clocks at any
//     N, one in TMEM 9 at N = 16, and shared memory's bandwidth is what bounds the tile.
//     The store to TMEM takes a quad's registers as four columns each, so the dims of a
//     column block lie there in another order (position 16 k + 4 q + e holds dim 16 q + 4
//     k + e), and those of Q's blocks with them;
//     What S^T reads from TMEM is handed over without a proxy fence (about 1,000
//     clocks); Q, in shared memory, is fenced in the first tile of a sequence, the
//     tile's copy in shared memory with P, before O^T;
//   * softmax: one token (= TMEM lane) a thread, the four warpgroups taking a quarter of
//     the heads each: s - m + 7 by one multiply-add, base 2 with a lazily moved maximum per head (a vote over the
//     warpgroup; O^T is rescaled only when a score exceeds the maximum by 2^8), P =
//     2^(s - m + 7) in FP16 (the offset uses FP16's upper range: weights down to 2^-21 of
//     the largest keep full precision); the row sums of the rounded P stay in registers
//     until the sequence ends.
// One warp issues S^T a pair of column blocks at a time as they arrive, and O^T per row
// block.  Separate warps for expanding and softmax, eight each, took longer: every step
// of the chain (expand, S^T, softmax, O^T) slows down, and there is no room in shared
// memory for a second tile that would let them overlap.
//
// Split: the batch's 128-token tiles form one flat range, cut equally over the CTAs of a
// head tile; a sequence's start (its Q, the last one's output) counts as one tile more
// (32 x 8,192 tokens, 16 heads: 35.1 us, 33.0 so).  A sequence that lies in one CTA is
// normalised and written there; others leave (m, l, O) partials that a second kernel
// joins.  Every wait is bounded.
//
// Measured (ragged lengths up to n, other pages each call): 32 sequences, n 8,192, 16 heads
// 34.0 us (30.1 where the pages lie in L2); 64, n 4,096, 64 heads 53.5 us; 8, n 32,768, 128
// heads 80.8 us (657 TFLOP/s); one of 77 tokens 7.4 us.  Of the first, in L2, some 4 us pass
// until the first tile is expanded, 19 us in nine tiles of 4,100 clocks, 7 us in storing and
// joining partials.  A tile is bound by its expansion (1,024
// conversions and as many packed multiplies a warp's width, 2,700 clocks with the stores)
// and by shared memory's bandwidth: 128 KB written and 150 KB (N 16) to 300 KB (N 64) of
// operands read at 128 bytes a clock.
#include <mutex>

#include "common.cuh"
#include "flat_plan.cuh"
#include "kernels.h"
#include "latent.cuh"
#include "quantize.cuh"
#include "tcgen05.cuh"

namespace nvfp4kv {

namespace {

constexpr int kWorkers = 512;                 // warps 0 .. 15
// The MMA warp is alone up to 32 heads (17 warps, 96 registers a thread).  With 64 it is the
// first of a warpgroup, whose other warps only meet the barriers, so that the working warps
// can take some of its registers: launched with 96 a thread, then 512 x 104 + 128 x 64 = 640
// x 96.  (A whole warpgroup with 16 or 32 heads: 32.2 against 30.9 us, 30.0 against 29.3.)
template <int N>
constexpr int kLThreads = kWorkers + (N == 64 ? 128 : 32);
constexpr int kWorkRegs = 104, kMmaRegs = 64;
static_assert(kWorkers * kWorkRegs + 128 * kMmaRegs <= kLThreads<64> * 96, "register split must fit the launch");
constexpr int kTile = 128;                    // tokens per tile
constexpr int kColBlock = kTile * 128;        // bytes of one column block (64 dims) of the tile
constexpr int kTileBytes = 8 * kColBlock;
constexpr uint32_t kWaitLimitL = 1u << 24;
constexpr float kNegInfL = -__builtin_huge_valf();
constexpr float kRescaleL = 8.0f;
constexpr int kSeqUnits = 1;                  // what a sequence's start costs a CTA, in tiles
constexpr float kPOffset = 7.0f;              // P = 2^(s - m + 7): at most 2^15
constexpr float kNoMax = 3.402823466e38f;     // the offset while every score was -inf: any other one moves the maximum, P of -inf is 0

template <int N>
struct LSmem {
    static constexpr int kSmemCbs = N == 64 ? 4 : 0;      // column blocks of S^T's A operand in shared memory (the first)
    static constexpr int kTmemCbs = 8 - kSmemCbs;         // ... and in TMEM
    static constexpr int kQBlock = N * 128;               // one column block of Q, [N][64]
    static constexpr int kQ = 0;                          // 8 FP16 blocks + the BF16 rotary block
    static constexpr int kKV = 9 * kQBlock;               // the tile
    static constexpr int kP = kKV + kTileBytes;           // FP16 [128 tokens][64], N heads used
    static constexpr int kBar = kP + kColBlock;
    static constexpr int kNumBars = 9;                    // kv_full[2] s_done p_full pv_done[4] drain
    static constexpr int kMisc = kBar + kNumBars * 8;     // tmem base, abort
    static constexpr int kM = (kMisc + 8 + 15) & ~15;     // float m[N], fac[N], alpha[N], off[N]
    static constexpr int kWarpMax = kM + 4 * N * 4;       // float [4][4][N / 4]: warps' maxima, and row sums at the end
    static constexpr int kBytes = kWarpMax + 4 * N * 4;
    // TMEM columns
    static constexpr uint32_t kColS = 4 * N, kColR = 5 * N, kColK = kColR + 32;   // O at 0
    static constexpr uint32_t kCols = 512;
    static_assert(kColK + 32 * kTmemCbs <= kCols, "TMEM columns");
    static_assert(kKV % 1024 == 0 && kP % 1024 == 0, "operand tiles need 1024-byte alignment");
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static_assert(sizeof(FlatScratch<kLThreads<N>>) <= kTileBytes, "the plan's scratch lies in the tile");
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

// Bounded wait that polls without suspending the thread (these waits are on the critical path).
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const volatile int *abort_flag) {
    for (uint32_t n = 0; n < kWaitLimitL; n++) {
        if (mbar_test_wait(bar, parity)) return true;
        if ((n & 63) == 63 && *abort_flag) return false;
    }
    return false;
}

// The tiles of a CTA's range in order.
struct TileIter {
    int b, t, nt, n;
    int left;       // units of the range from this one on
};

__device__ __forceinline__ void set_seq(const LatentArgs &a, TileIter &it) {
    it.n = clamp_rows(__ldg(a.seq_lens + it.b), a.cap);
    it.nt = (it.n + kTile - 1) / kTile;
}

__device__ __forceinline__ void next_tile(const LatentArgs &a, TileIter &it) {
    it.left--;
    if (++it.t < it.nt || it.left <= 0) return;
    it.t = 0;
    it.left -= kSeqUnits;
    if (it.left <= 0) return;
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

// Barriers 1 .. 4: the working warpgroups; 5: all of them.
__device__ __forceinline__ void group_sync(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); }
__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 5, 512;" ::: "memory"); }

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

// v[c] (c < CW <= 16) summed over the warp's lanes: lane c returns column c's sum (lanes >= CW: a copy of c % CW's)
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

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ int seq_tiles(const LatentArgs &a, int b) {
    return (clamp_rows(__ldg(a.seq_lens + b), a.cap) + kTile - 1) / kTile;
}

// Units of sequence b in the flat order: its tiles, after kSeqUnits that stand for its start.
__device__ __forceinline__ unsigned seq_units(const LatentArgs &a, int b) {
    const int nt = seq_tiles(a, b);
    return nt ? nt + kSeqUnits : 0;
}

template <int N>
__global__ void __launch_bounds__(kLThreads<N>, 1) latent_decode_kernel(LatentArgs a) {
    using L = LSmem<N>;
    constexpr int CW = N / 4;                     // heads per warpgroup
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBar);
    uint64_t *kv_full = bars, *s_done = bars + 2, *p_full = bars + 3, *pv_done = bars + 4, *drain = bars + 8;
    uint32_t &tmem_base = *reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    float *s_m = reinterpret_cast<float *>(smem + L::kM), *s_fac = s_m + N, *s_alpha = s_fac + N, *s_off = s_alpha + N;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h0 = blockIdx.y * N;
    if (tid == 0) {
        for (int i = 0; i < L::kNumBars; i++)
            mbar_init(&bars[i], i < 2 || i == 3 ? kWorkers / 32 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait();               // everything read or written may belong to earlier work of the stream
    pdl_launch_dependents();
    if (warp == 16) tc_alloc(&tmem_base, L::kCols);   // (after the wait: an earlier kernel may need the columns first)

    int b0;
    unsigned first, u0 = 0, u1 = 0;
    flat_locate<kLThreads<N>>(
        *reinterpret_cast<FlatScratch<kLThreads<N>> *>(smem + L::kKV), a.B, [&](int b) { return seq_units(a, b); },
        [&](unsigned total) {
            const FlatCut cut(total, a.splits);
            u0 = cut.begin(blockIdx.x);
            u1 = cut.begin(blockIdx.x + 1);
            return u0 < u1 ? u0 : kFlatNone;
        },
        b0, first);
    if (warp == 16) {   // lengths out of range, and the rows of sequences of length 0
        for (int b = blockIdx.x; b < a.B; b += a.splits) {
            const int32_t n = __ldg(a.seq_lens + b);
            if (lane == 0 && blockIdx.y == 0 && (n < 0 || (int64_t)n > a.cap)) flag_error(a.err, kErrSeqLen);
            if (n > 0) continue;
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + ((int64_t)b * a.H + h0) * kLatentDim);
            for (int i = lane; i < min(N, a.H - h0) * (kLatentDim / 8); i += 32) dst[i] = make_uint4(0, 0, 0, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    TileIter it;
    it.b = b0;
    it.t = max(0, (int)(u0 - first) - kSeqUnits);
    it.left = (int)(u1 - u0) - max(0, (int)(first + kSeqUnits - u0));
    if (u0 >= u1 || it.left <= 0) {   // a range without tiles
        if (warp == 16) tc_dealloc(tmem_base, L::kCols);
        return;
    }
    set_seq(a, it);
    const uint32_t tmem = tmem_base, sbase = smem_u32(smem);
    if (warp >= 16) {
        // ---------------- the MMA warp
        // The whole warp runs the loop and one elected lane issues, so that the compiler
        // sees the descriptors as uniform values: a product issued under a divergent
        // branch cost 70 to 110 clocks, more than the products themselves (38 at N = 16,
        // 47 at N = 64).
        if (N == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
        if (warp == 16) {
            constexpr uint32_t idesc_s = idesc_f16_f32(128, N, false), idesc_r = idesc_bf16_f32(128, N, false);
            constexpr uint32_t idesc_o = idesc_a_mn_major(idesc_f16_f32(128, N, true));
            auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
            const uint32_t tm = uniform(tmem);
            const bool leader = elect_one();
            // operand descriptors; a step adds its byte offset / 16 to the address field
            const uint64_t dC = smem_desc_sw128(sbase + L::kKV, 16, 1024), dQ = smem_desc_sw128(sbase + L::kQ, 16, 1024);
            const uint64_t dP = smem_desc_sw128(sbase + L::kP, 16, 1024), dV = smem_desc_sw128(sbase + L::kKV, kColBlock, 1024);
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                const bool good = __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
                tc_fence_after();
                return good;
            };
            bool fresh = true, ok = true;   // fresh: the tile is the range's first of its sequence
            for (uint32_t j = 0; it.left > 0; j++) {
                // (unrolled by 1, 2 and 4: 32 sequences, n 8,192, 16 heads 30.9, 29.6 and 30.4 us; 8, n 32,768,
                // 128 heads 85.9, 81.1 and 80.6)
#pragma unroll(N == 64 ? 4 : 2)
                for (uint32_t i = 0; i < 4; i++) {   // column blocks 2 i, 2 i + 1 (and the rotary part, with the first)
                    if (!(i & 1)) ok = ok && wait(&kv_full[i >> 1], j & 1);
                    if (!ok) break;
                    const uint64_t q = dQ + i * (2 * L::kQBlock / 16), c = dC + i * (2 * kColBlock / 16);
                    const uint32_t t = tm + L::kColK + 32 * (2 * i - L::kSmemCbs);
                    if (leader) {
                        if (i == 0) {
#pragma unroll
                            for (int kk = 0; kk < 4; kk++)
                                tc_mma_bf16_tmem_a(tm + L::kColS, tm + L::kColR + kk * 8, dQ + (8 * L::kQBlock / 16 + kk * 2),
                                                   idesc_r, kk > 0);
                        }
                        if (L::kSmemCbs == 0 || 2 * i >= L::kSmemCbs) {
#pragma unroll
                            for (int kk = 0; kk < 8; kk++)
                                tc_mma_bf16_tmem_a(tm + L::kColS, t + kk * 8,
                                                   q + ((kk >> 2) * (L::kQBlock / 16) + (kk & 3) * 2), idesc_s, 1u);
                        } else {
#pragma unroll
                            for (int kk = 0; kk < 8; kk++)
                                tc_mma_bf16(tm + L::kColS, c + ((kk >> 2) * (kColBlock / 16) + (kk & 3) * 2),
                                            q + ((kk >> 2) * (L::kQBlock / 16) + (kk & 3) * 2), idesc_s, 1u);
                        }
                        if (i == 3) tc_commit(s_done);
                    }
                }
                ok = ok && wait(p_full, j & 1);
                if (!ok) break;
                if (leader) {
                    const uint32_t acc = fresh ? 0u : 1u;
#pragma unroll 1
                    for (uint32_t mb = 0; mb < 4; mb++) {
                        const uint64_t v = dV + mb * (2 * kColBlock / 16);
#pragma unroll
                        for (int kk = 0; kk < 8; kk++)   // 16 tokens: 2,048 bytes of a column block, and of P
                            tc_mma_bf16(tm + mb * N, v + kk * 128, dP + kk * 128, idesc_o, kk > 0 ? 1u : acc);
                        tc_commit(&pv_done[mb]);
                    }
                }
                const int b = it.b;
                next_tile(a, it);
                fresh = it.b != b;
            }
            if (!ok && leader) {
                if (!*abort_flag) flag_error(a.err, kErrTimeout);
                *abort_flag = 1;
                tc_commit(drain);   // no product may still read the CTA's memory when it ends
                mbar_wait_bounded(drain, 0, kWaitLimitL, nullptr);
            }
        }
        __syncwarp();
    } else {
        // ---------------- expanding and softmax
        // A wait that gave up sets the abort flag, which ends every other wait; the
        // warps then still run through their tiles (on meaningless values), so that
        // no barrier is left short of a warp.
        if (N == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWorkRegs));
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!wait_bar(bar, parity, abort_flag) && !*abort_flag) {
                *abort_flag = 1;
                flag_error(a.err, kErrTimeout);
            }
            __syncwarp();
        };
        const int wg = warp >> 2, row = 32 * (warp & 3) + lane;   // softmax: head quarter, token
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        // expanding: group grp of the tile (its TMEM lanes are this warp's to reach), column blocks 2 i + par, rows
        // er and er + 8, 16-value block eq of a column block
        const int grp = 2 * (warp & 3) + (wg & 1), par = wg >> 1, er = lane >> 2, eq = lane & 3;
        const uint32_t glanes = (uint32_t)(16 * grp) << 16;
        uint2 raw[4][2];
        uint4 scl[2], rope[2];
        auto page_of = [&](const TileIter &x) -> int32_t {        // page of the group (-1: none)
            const int t = x.t * kTile + 16 * grp;
            if (x.left <= 0 || t >= x.n) return -1;
            return __ldg(a.block_table + (int64_t)x.b * a.max_pages + (t >> a.log2P));
        };
        // the group's address and how many of its rows exist (0: none, or a page out of range, flagged)
        auto group_of = [&](const TileIter &x, int32_t page, int &rows) -> const uint8_t * {
            const int t = x.t * kTile + 16 * grp;
            rows = x.left > 0 ? x.n - t : 0;
            if (rows > 0 && (page < 0 || page >= a.num_pages)) {
                if (lane == 0) flag_error(a.err, kErrPage);
                rows = 0;
            }
            return a.pool + (int64_t)(rows > 0 ? page : 0) * ((int64_t)kLatentRow * a.P) +
                   (int64_t)((t & (a.P - 1)) >> 4) * kLatentGroup;
        };
        auto load_block = [&](const uint8_t *p, int rows, int i) {
#pragma unroll
            for (int e = 0; e < 2; e++)
                raw[i][e] = er + 8 * e < rows
                                ? __ldg(reinterpret_cast<const uint2 *>(p + (2 * i + par) * 512 + (er + 8 * e) * 32 + eq * 8))
                                : make_uint2(0, 0);
        };
        auto load_scales = [&](const uint8_t *p, int rows) {      // byte 2 cb + eq % 2: of column block cb
#pragma unroll
            for (int e = 0; e < 2; e++)
                scl[e] = er + 8 * e < rows
                             ? __ldg(reinterpret_cast<const uint4 *>(p + kLatentScales + (er + 8 * e) * 32 + (eq >> 1) * 16))
                             : make_uint4(0, 0, 0, 0);
        };
        auto load_rope = [&](const uint8_t *p, int rows) {        // 16-byte chunk 4 par + eq
#pragma unroll
            for (int e = 0; e < 2; e++)
                rope[e] = er + 8 * e < rows ? __ldg(reinterpret_cast<const uint4 *>(
                                                  p + kLatentRope + (er + 8 * e) * 128 + (((4 * par + eq) ^ er) << 4)))
                                            : make_uint4(0, 0, 0, 0);
        };
        // Q of sequence b: a warp per head (N / 16 heads each), FP16 latent blocks and the BF16 rotary
        // block, requested two heads at a time (the next tile's bytes hold the registers).
        constexpr int QH = N / (kWorkers / 32), QB = QH < 2 ? QH : 2;
        auto fetch_q = [&](int b, int k0, auto &qv, auto &qx) {
#pragma unroll
            for (int k = 0; k < (int)(sizeof(qx) / 4); k++) {
                const int h = h0 + warp + (k0 + k) * (kWorkers / 32);
                qv[k][0] = qv[k][1] = make_uint4(0, 0, 0, 0);
                qx[k] = 0;
                if (h < a.H) {
                    const int64_t at = (int64_t)b * a.H + h;
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.ql + at * kLatentDim) + lane * 2;
                    qv[k][0] = __ldg(src);
                    qv[k][1] = __ldg(src + 1);
                    qx[k] = __ldg(reinterpret_cast<const uint32_t *>(a.qr + at * kRopeDim) + lane);
                }
            }
        };
        auto prefetch_q = [&](int b) {          // to L2, the whole tile's heads: 128-byte lines, one a thread
            const int lines = min(N, a.H - h0) * 8;
            for (int i = tid; i < lines; i += kWorkers)
                prefetch_l2(a.ql + ((int64_t)b * a.H + h0) * kLatentDim + 64 * i);
            if (tid < lines / 8) prefetch_l2(a.qr + ((int64_t)b * a.H + h0 + tid) * kRopeDim);
        };
        // (The previous sequence's S^T are done: its scores were seen.)
        auto store_q = [&](int k0, auto &qv, auto &qx) {
#pragma unroll
            for (int k = 0; k < (int)(sizeof(qx) / 4); k++) {
                const int hh = warp + (k0 + k) * (kWorkers / 32);
                const uint4 x0 = qv[k][0], x1 = qv[k][1];
                const uint32_t xr = qx[k];
                const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                uint32_t ml = 0, mr = xr & 0x7fff7fffu;
#pragma unroll
                for (int e = 0; e < 8; e++) ml = max_u16x2(ml, w[e] & 0x7fff7fffu);
                ml = __reduce_max_sync(0xffffffffu, max(ml >> 16, ml & 0xffffu));
                mr = __reduce_max_sync(0xffffffffu, max(mr >> 16, mr & 0xffffu));
                // 2^kq puts the largest |q g| into [2^14, 2^15), but enlarges the rotary part to 2^64 at
                // most: its products with keys below 2^57, 64 of them, stay in FP32 (a latent part that
                // loses bits in FP16 then is below 2^-77 of the rotary one)
                const uint32_t top = __float_as_uint(__uint_as_float(ml << 16) * a.g);
                int kq = top ? 14 - ((int)(top >> 23) - 127) : 0;
                kq = max(-126, min(min(126, kq), max(0, 63 - ((int)(mr >> 7) - 127))));
                const float sc = __uint_as_float((uint32_t)(kq + 127) << 23);
                uint32_t f[8];
#pragma unroll
                for (int e = 0; e < 8; e++) f[e] = f32x2_to_f16x2(bf16_hi(w[e]) * a.g * sc, bf16_lo(w[e]) * a.g * sc);
                uint8_t *q = smem + L::kQ + (lane >> 2) * L::kQBlock;      // lane: dims 16 lane .. 16 lane + 15
                const int bq = lane & 3;
                if ((lane >> 2) >= L::kSmemCbs) {   // in the order of the block in TMEM
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        *reinterpret_cast<uint2 *>(q + sw128_off(hh, 2 * k + (bq >> 1)) + (bq & 1) * 8) =
                            make_uint2(f[2 * k], f[2 * k + 1]);
                } else {
                    *reinterpret_cast<uint4 *>(q + sw128_off(hh, bq * 2)) = make_uint4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<uint4 *>(q + sw128_off(hh, bq * 2 + 1)) = make_uint4(f[4], f[5], f[6], f[7]);
                }
                // rotary dims 32 p + 8 q + 4 k + e (here d = 2 lane, + 1) at position 32 p + 16 k + 4 q + e
                const int d = 2 * lane, pos = (d & 32) + ((d >> 2) & 1) * 16 + ((d >> 3) & 3) * 4 + (d & 3);
                *reinterpret_cast<uint32_t *>(smem + L::kQ + 8 * L::kQBlock + sw128_off(hh, pos >> 3) + (pos & 7) * 2) =
                    f32x2_to_bf16x2(bf16_hi(xr) * sc, bf16_lo(xr) * sc);
                if (lane == 0) {
                    s_fac[hh] = a.score_log2 * __uint_as_float((uint32_t)(127 - kq) << 23);
                    s_m[hh] = kNegInfL;
                    s_off[hh] = kNoMax;
                }
            }
        };
        auto load_q = [&]() {   // (handed to the tensor core with the first half of the tile)
            uint4 qv[QB][2];
            uint32_t qx[QB];
#pragma unroll 1
            for (int k0 = 0; k0 < QH; k0 += QB) {
                fetch_q(it.b, k0, qv, qx);
                store_q(k0, qv, qx);
            }
            workers_sync();   // s_fac and s_m are written for all heads
        };
        auto load_tile = [&](const uint8_t *p, int rows) {
            load_scales(p, rows);
#pragma unroll
            for (int i = 0; i < 4; i++) load_block(p, rows, i);
            load_rope(p, rows);
        };
        TileIter nx = it;                       // the tile whose bytes are requested next
        {   // the first tile and the first sequence's Q
            uint4 qv[QH][2];
            uint32_t qx[QH];
            const int32_t page = page_of(nx);
            fetch_q(it.b, 0, qv, qx);
            int rows;
            const uint8_t *p = group_of(nx, page, rows);
            if (QB < QH) {   // the tile's bytes come to L2 while Q, which needs the registers, is laid out
                if (rows > 0 && par == 0 && lane < kLatentGroup / 256) {
                    prefetch_l2(p + lane * 256);
                    prefetch_l2(p + lane * 256 + 128);
                }
                store_q(0, qv, qx);
                load_tile(p, rows);
            } else {
                load_tile(p, rows);
                store_q(0, qv, qx);
            }
            workers_sync();   // s_fac and s_m are written for all heads
        }
        next_tile(a, nx);
        int32_t npage = page_of(nx);            // its page, requested a tile earlier still
        // With 64 heads a tile the bytes of the tile after that are brought to L2 (64 sequences of up to
        // 4,096 tokens: 58.1 us without, 56.1 so; with 16 heads it costs what it gains).
        constexpr bool kAhead = N == 64;
        TileIter pf = nx;
        int32_t ppage = -1;
        if (kAhead) {
            if (pf.left > 0) next_tile(a, pf);
            ppage = page_of(pf);
        }
        bool fresh = true;                      // the range's first tile of its sequence
        int t_begin = it.t;
        float l[CW];
        for (uint32_t j = 0; it.left > 0; j++) {
            if (fresh) {
                if (j > 0) load_q();
#pragma unroll
                for (int c = 0; c < CW; c++) l[c] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {       // ---- expand block eq of column block 2 i + par, rows er and er + 8
                uint32_t f[2][8];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const uint32_t sw = i == 0 ? scl[e].x : i == 1 ? scl[e].y : i == 2 ? scl[e].z : scl[e].w;
                    const uint32_t sb = (sw >> (16 * par + 8 * (eq & 1))) & 0xffu;
                    const uint32_t s = e4m3x2_to_f16x2(sb * 0x101u);
                    e2m1x8_to_f16x2x4(raw[i][e].x, f[e][0], f[e][1], f[e][2], f[e][3]);
                    e2m1x8_to_f16x2x4(raw[i][e].y, f[e][4], f[e][5], f[e][6], f[e][7]);
#pragma unroll
                    for (int x = 0; x < 8; x++) f[e][x] = hmul2(f[e][x], s);
                }
                // (TMEM's copy is free: the previous tile's scores were seen)
                if (2 * i >= L::kSmemCbs) {
                    const uint32_t st[16] = {f[0][0], f[0][1], f[1][0], f[1][1], f[0][2], f[0][3], f[1][2], f[1][3],
                                             f[0][4], f[0][5], f[1][4], f[1][5], f[0][6], f[0][7], f[1][6], f[1][7]};
                    tc_st_16x256_x4(tmem + glanes + L::kColK + 32 * (2 * i + par - L::kSmemCbs), st);
                }
                if (i == 0) {
                    const uint32_t st[8] = {rope[0].x, rope[0].y, rope[1].x, rope[1].y, rope[0].z, rope[0].w, rope[1].z, rope[1].w};
                    tc_st_16x256_x2(tmem + glanes + L::kColR + 16 * par, st);
                }
                if (j > 0) wait(&pv_done[i], (j - 1) & 1);
                uint8_t *blk = smem + L::kKV + (2 * i + par) * kColBlock;
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int tr = 16 * grp + er + 8 * e;
                    *reinterpret_cast<uint4 *>(blk + sw128_off(tr, 2 * eq)) = make_uint4(f[e][0], f[e][1], f[e][2], f[e][3]);
                    *reinterpret_cast<uint4 *>(blk + sw128_off(tr, 2 * eq + 1)) = make_uint4(f[e][4], f[e][5], f[e][6], f[e][7]);
                }
                if (i & 1) {   // half of the tile at a time (a quarter at a time: the same)
                    // S^T reads shared memory through the async proxy: the column blocks that lie there, and Q,
                    // which a sequence's first tile hands over with the first half
                    if (2 * i <= L::kSmemCbs || (i == 1 && fresh)) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&kv_full[i >> 1]);
                }
            }
            // Request the next tile's bytes, and the page after that.  Only here: a proxy fence waits
            // for loads in flight, and the next one follows the softmax.
            {
                int rows;
                const uint8_t *p = group_of(nx, npage, rows);
                load_tile(p, rows);
                if (kAhead) {
                    if (par == 0 && ppage >= 0 && ppage < a.num_pages && lane < kLatentGroup / 256) {
                        const uint8_t *group = a.pool + (int64_t)ppage * ((int64_t)kLatentRow * a.P) +
                                               (int64_t)(((pf.t * kTile + 16 * grp) & (a.P - 1)) >> 4) * kLatentGroup;
                        prefetch_l2(group + lane * 256);
                        prefetch_l2(group + lane * 256 + 128);
                    }
                    nx = pf;
                    npage = ppage;
                    if (pf.left > 0) next_tile(a, pf);
                    ppage = page_of(pf);
                } else {
                    next_tile(a, nx);
                    npage = page_of(nx);
                }
            }
            // ---- softmax of the token's scores for the warpgroup's heads.  S^T done says that the
            // previous tile's O^T, issued before it, is done too: P and O^T may be written.
            if (warp == 0) wait(s_done, j & 1);   // one warp polls: sixteen would take shared memory's time from S^T
            workers_sync();
            tc_fence_after();
            const bool seen = it.t * kTile + row < it.n;
            // d = s - m + 7, one multiply-add with the head's factor and offset 7 - m, read from TMEM in
            // chunks of up to eight heads (the next tile's bytes hold the registers): once to see whether
            // a maximum must move, and with more heads a thread again to form P.
            constexpr int CH = CW < 8 ? CW : 8;
            auto load_diffs = [&](int c0, float (&d)[CH]) {
                uint32_t sr[CH];
                tc_ld(tmem + lanes + L::kColS + wg * CW + c0, sr);
                const float4 *fac = reinterpret_cast<const float4 *>(s_fac + wg * CW + c0);
                const float4 *off = reinterpret_cast<const float4 *>(s_off + wg * CW + c0);
                tc_wait_ld();
#pragma unroll
                for (int x = 0; x < CH / 4; x++) {
                    const float4 f = fac[x], o = off[x];
                    d[4 * x] = fmaf(__uint_as_float(sr[4 * x]), f.x, o.x);
                    d[4 * x + 1] = fmaf(__uint_as_float(sr[4 * x + 1]), f.y, o.y);
                    d[4 * x + 2] = fmaf(__uint_as_float(sr[4 * x + 2]), f.z, o.z);
                    d[4 * x + 3] = fmaf(__uint_as_float(sr[4 * x + 3]), f.w, o.w);
                }
                if (!seen) {
#pragma unroll
                    for (int c = 0; c < CH; c++) d[c] = kNegInfL;
                }
            };
            float d[CH], top = kNegInfL;
#pragma unroll
            for (int c0 = 0; c0 < CW; c0 += CH) {
                load_diffs(c0, d);
#pragma unroll
                for (int c = 0; c < CH; c++) top = fmaxf(top, d[c]);
            }
            const bool moves = group_any(wg, top > kRescaleL + kPOffset);
            if (moves) {
                float *wmax = reinterpret_cast<float *>(smem + L::kWarpMax) + wg * 4 * CW;
                int mine = 0;
#pragma unroll
                for (int c0 = 0; c0 < CW; c0 += CH) {
                    uint32_t sr[CH];
                    tc_ld(tmem + lanes + L::kColS + wg * CW + c0, sr);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < CH; c++) {
                        const float sc = seen ? __uint_as_float(sr[c]) * s_fac[wg * CW + c0 + c] : kNegInfL;
                        const int mx = __reduce_max_sync(0xffffffffu, ordered(sc));
                        if (lane == c0 + c) mine = mx;
                    }
                }
                if (lane < CW) wmax[(warp & 3) * CW + lane] = unordered(mine);
                group_sync(wg);
                if ((warp & 3) == 0 && lane < CW) {
                    const float mx = fmaxf(fmaxf(wmax[lane], wmax[CW + lane]), fmaxf(wmax[2 * CW + lane], wmax[3 * CW + lane]));
                    const float mo = s_m[wg * CW + lane], mn = fmaxf(mo, mx);
                    s_alpha[wg * CW + lane] = mo == kNegInfL ? 0.f : ex2(mo - mn);
                    s_m[wg * CW + lane] = mn;
                    s_off[wg * CW + lane] = mn == kNegInfL ? kNoMax : kPOffset - mn;
                }
                group_sync(wg);
#pragma unroll
                for (int c = 0; c < CW; c++) l[c] *= s_alpha[wg * CW + c];
                if (!fresh) {   // O^T holds the earlier tiles: rescale the warpgroup's heads
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
            if (CW == CH && moves) load_diffs(0, d);
#pragma unroll
            for (int c0 = 0; c0 < CW; c0 += CH) {
                if (CW > CH) load_diffs(c0, d);
                uint32_t pw[CH / 2];
#pragma unroll
                for (int e = 0; e < CH / 2; e++) {
                    pw[e] = f32x2_to_f16x2(ex2(d[2 * e + 1]), ex2(d[2 * e]));
                    add_f16x2(l[c0 + 2 * e], l[c0 + 2 * e + 1], pw[e]);
                }
                if (CW == 4)   // eight bytes a thread: two warpgroups share a 16-byte chunk
                    *reinterpret_cast<uint2 *>(smem + L::kP + sw128_off(row, wg >> 1) + (wg & 1) * 8) = make_uint2(pw[0], pw[1]);
                else
                    *reinterpret_cast<uint4 *>(smem + L::kP + sw128_off(row, (wg * CW + c0) / 8)) =
                        make_uint4(pw[0], pw[1], pw[CH / 2 - 2], pw[CH / 2 - 1]);
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
            if (it.left > 0) prefetch_q(it.b);
#pragma unroll 1
            for (int i = 0; i < 4; i++) wait(&pv_done[i], j & 1);
            tc_fence_after();
            {
                float *wsum = reinterpret_cast<float *>(smem + L::kWarpMax) + wg * 4 * CW;
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
                const int hw = h0 + wg * CW, nh = a.H - hw;     // the warpgroup's first head, and how many there are
                if (whole) {
                    float inv[CW];
#pragma unroll
                    for (int c = 0; c < CW; c++)
                        inv[c] = a.g / ((wsum[c] + wsum[CW + c]) + (wsum[2 * CW + c] + wsum[3 * CW + c]));
                    __nv_bfloat16 *dst = a.out + ((int64_t)cur.b * a.H + hw) * kLatentDim + row;
#pragma unroll 1
                    for (int mb = 0; mb < 4; mb++, dst += 128) {
                        uint32_t ov[CW];
                        tc_ld(tmem + lanes + mb * N + wg * CW, ov);
                        tc_wait_ld();
#pragma unroll
                        for (int c = 0; c < CW; c++)
                            if (c < nh) dst[c * kLatentDim] = __float2bfloat16_rn(__uint_as_float(ov[c]) * inv[c]);
                    }
                } else {
                    float *dst = a.part_acc + (slot * a.H + hw) * kLatentDim + row;
#pragma unroll 1
                    for (int mb = 0; mb < 4; mb++, dst += 128) {
                        uint32_t ov[CW];
                        tc_ld(tmem + lanes + mb * N + wg * CW, ov);
                        tc_wait_ld();
#pragma unroll
                        for (int c = 0; c < CW; c++)
                            if (c < nh) dst[c * kLatentDim] = __uint_as_float(ov[c]);
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
    if (warp == 16) tc_dealloc(tmem, L::kCols);
}

// Joins the partials of the sequences that several CTAs covered: one CTA per (sequence,
// head), thread t of a group of 128 owns dims 4 t .. 4 t + 3, and the groups (as many as
// the launch has) take the partials in turn, U at a time.  It waits for loads: U and the
// groups are as large as one wave of CTAs allows (8 x 128 heads, 11 partials on average:
// 4.9 us with U = 8, 8.7 us with U = 4 and four groups in two waves).
constexpr int kJoinGroup = 128, kJoinGroups = 8, kJoinWave = 152 * 8;   // groups of threads that run at once

template <int U>
__global__ void __launch_bounds__(kJoinGroup *kJoinGroups) latent_join_kernel(LatentArgs a) {
    __shared__ unsigned s_sum[2][kJoinGroup * kJoinGroups / 32];
    __shared__ float2 s_ml[kJoinGroups];
    __shared__ float4 s_acc[kJoinGroups - 1][kJoinGroup];
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, t = tid & (kJoinGroup - 1), grp = tid / kJoinGroup;
    const int groups = blockDim.x / kJoinGroup;
    // The lengths may be read before the wait: the decode kernel lets this one start only
    // after its own wait for everything before it, and does not write them.
    const int nt = seq_tiles(a, b);
    unsigned before = 0, all = 0;
    for (int x = tid; x < a.B; x += blockDim.x) {
        const unsigned n = seq_units(a, x);
        all += n;
        if (x < b) before += n;
    }
    all = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, before);
    if ((tid & 31) == 0) {
        s_sum[0][tid >> 5] = all;
        s_sum[1][tid >> 5] = before;
    }
    __syncthreads();
    all = before = 0;
    for (int w = 0; w < (int)blockDim.x / 32; w++) {
        all += s_sum[0][w];
        before += s_sum[1][w];
    }
    pdl_wait();
    if (nt == 0) return;    // zeroed already
    const FlatCut cut(all, a.splits);
    const int c0 = cut.piece(before + kSeqUnits), c1 = cut.piece(before + kSeqUnits + nt - 1);
    if (c0 == c1) return;   // written by its CTA
    float m = kNegInfL, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0 + grp; c <= c1; c += U * groups) {
        float2 ml[U];
        float4 v[U];
#pragma unroll
        for (int k = 0; k < U; k++) {
            ml[k] = make_float2(kNegInfL, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + k * groups <= c1) {
                const int64_t at = (int64_t)(c + k * groups + b) * a.H + h;
                ml[k] = __ldcg(a.part_ml + at);
                v[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_acc + at * kLatentDim) + t);
            }
        }
        float mx = m;
#pragma unroll
        for (int k = 0; k < U; k++) mx = fmaxf(mx, ml[k].x);
        const float f0 = m == kNegInfL ? 0.f : ex2(m - mx);
        l *= f0;
        acc.x *= f0;
        acc.y *= f0;
        acc.z *= f0;
        acc.w *= f0;
#pragma unroll
        for (int k = 0; k < U; k++) {
            const float f = ml[k].x == kNegInfL ? 0.f : ex2(ml[k].x - mx);
            l += f * ml[k].y;
            acc.x += f * v[k].x;
            acc.y += f * v[k].y;
            acc.z += f * v[k].z;
            acc.w += f * v[k].w;
        }
        m = mx;
    }
    if (groups > 1) {
        if (t == 0) s_ml[grp] = make_float2(m, l);
        if (grp > 0) s_acc[grp - 1][t] = acc;
        __syncthreads();
        if (grp > 0) return;
        float mx = m;
        for (int g = 1; g < groups; g++) mx = fmaxf(mx, s_ml[g].x);
        const float f0 = m == kNegInfL ? 0.f : ex2(m - mx);
        l *= f0;
        acc.x *= f0;
        acc.y *= f0;
        acc.z *= f0;
        acc.w *= f0;
        for (int g = 1; g < groups; g++) {
            const float2 o = s_ml[g];
            if (o.x == kNegInfL) continue;
            const float f = ex2(o.x - mx);
            const float4 v = s_acc[g - 1][t];
            l += f * o.y;
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
        }
    }
    const float inv = a.g / l;
    reinterpret_cast<uint2 *>(a.out + ((int64_t)b * a.H + h) * kLatentDim)[t] =
        make_uint2(f32x2_to_bf16x2(acc.y * inv, acc.x * inv), f32x2_to_bf16x2(acc.w * inv, acc.z * inv));
}

// Heads of a CTA's tile.  More of them share an expanded tile: 32 sequences of 4,096 tokens
// take 29.9 us with 32 heads in one tile and 41.6 us in two of 16, 41.3 us with 64 heads in
// one tile and 49.8 us in two of 32 (69.5 against 87.7 us with 128 heads).
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

namespace {

cudaError_t sm_count(int *sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevicesL)) e = cudaErrorInvalidDevice;
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_mu_l);
    if (!g_sms_l[dev]) e = cudaDeviceGetAttribute(&g_sms_l[dev], cudaDevAttrMultiProcessorCount, dev);
    *sms = g_sms_l[dev];
    return e;
}

}  // namespace

int latent_decode_auto_splits(int num_heads, cudaError_t *status) {
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
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
    int dev = 0, smem = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    // No more CTAs than there can be token tiles; and while there are SMs for it, smaller head
    // tiles, whose steps are shorter (200 tokens: 9.6 us instead of 14.3 with 64 or 128 heads).
    // Both, and whether a join follows, go by the table's width: the lengths are on the device.
    const int64_t cap = (int64_t)max_pages * c.page_size, most = batch * ((cap + kTile - 1) / kTile);
    int n = tile_heads(num_heads);
    for (int x = 16; x < n; x *= 2)
        if (most * ((num_heads + x - 1) / x) <= sms) n = x;
    const int tiles = (num_heads + n - 1) / n;
    if (splits > most) splits = (int)most;
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
    a.cap = cap;
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
    e = launch_pdl(fn, dim3((unsigned)splits, (unsigned)tiles), n == 64 ? kLThreads<64> : kLThreads<16>, (size_t)smem, stream, args);
    if (e != cudaSuccess || splits == 1 || a.cap <= kTile) return e;   // no sequence can have been split
    // The partials of a sequence of the batch's average length
    const int partials = (splits + batch - 1) / batch + 1;
    int groups = 1;
    while (groups < kJoinGroups && groups * 8 < partials && (int64_t)batch * num_heads * groups * 2 <= kJoinWave) groups *= 2;
    return launch_pdl(partials <= 4 ? reinterpret_cast<const void *>(&latent_join_kernel<4>)
                                    : reinterpret_cast<const void *>(&latent_join_kernel<8>),
                      dim3((unsigned)num_heads, (unsigned)batch), (unsigned)(kJoinGroup * groups), 0, stream, args);
}

}  // namespace nvfp4kv
