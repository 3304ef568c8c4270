// tree_attention.cu -- attention of each sequence's drafted tokens over the paged NVFP4 cache.
//
// The last d cached tokens of a sequence (its drafts, in the pages like the rest) form a tree:
// draft i sees the base = n - d tokens before the drafts and, of the drafts, those that its
// mask names (its ancestors and itself).  Its position is base + popcount(mask_i) - 1, the one
// that its rotation used.  With s = sm_scale g_K q . k:
//   z = cap tanh(s / cap) (or s),   z += slope_h (pos_key - pos_i),   only keys with
//   pos_key > pos_i - window,   out = g_V softmax(z) V.
// One draft and no options: decode attention.  The rows of a (sequence, kv head) pair are its
// d x G queries, row = i G + head of the group: they share every K and V row.
//
// A token costs 144 bytes a kv head and 512 flops a row: the cache's bytes bound it up to some
// 128 rows, the tensor cores beyond.
//
// Tokens sit on the tensor core's M dimension in both products, rows on N (16, 32, 64 or 128),
// so few rows cost little:
//   S^T (128 tokens x N) = K Q^T     8 steps of M 128 x N x K 16, K as the A operand in TMEM
//   O^T (128 dims x N) += V^T P^T    8 steps, V and P in shared memory, both MN-major
// e2m1 x e4m3 is an exact FP16 value.  Q is FP16 after a power-of-two pre-scale a row (exact
// above 2^-29 of the row's largest value); the tensor scales go into the score's factor and
// into the output.
//
// Warps:
//   * eight workers (sixteen with 128 rows) expand a tile and run its softmax.  Expanding: a
//     warp takes a 16-token group, K and V (with 128 rows one of them); lane (r, q) holds the
//     q-th 16 bytes of rows r and r + 8.  K goes to TMEM (the store takes a quad's registers as
//     four columns each, so the dims lie there in another order: position 16 a + 4 q + e holds
//     dim 32 q + 4 a + e, and Q's with them), V to a swizzled tile in shared memory.  Softmax:
//     one token (= TMEM lane) a thread, the warpgroups sharing the rows; a lazily moved maximum
//     per row (a vote over the warpgroup; O^T is rescaled only when a score exceeds it by 2^8),
//     P = 2^(z - m + 7) in FP16 (the offset uses FP16's upper range), the sums of the rounded P
//     in registers until the pair ends.  Options and masks change the scores in TMEM before
//     that, in tiles that have any.
//   * one warp copies raw tiles (8 groups of 2,304 bytes) into a ring, ahead of everything;
//   * one warp issues the products.
// Up to 64 rows two CTAs share an SM.  K of tile j + 1 is expanded while the products of tile j
// - 1 run; O^T += V^T P^T of a tile and S^T of the next are handed over together and awaited
// together, so that a tile costs two waits and one vote.  The chain of a tile (K, wait, V,
// softmax, products) is long beside its instructions: the other CTA fills the gaps.  With 128
// rows O^T and S^T leave no TMEM for a second CTA: one, with S double and V triple, so
// that S^T of tile j + 1 runs during the softmax of tile j.
//
// Measured (ragged lengths up to n, 64 query and 8 kv heads, cold L2): 16 sequences, n 32,768, 1
// draft (8 rows) 115 us, 4 drafts (32 rows) 129, 8 (64 rows) 176, 16 (128 rows) 302: 470
// TFLOP/s.  A tile takes an SM some 1,250, 1,350, 2,000 and 3,700 clocks (its bytes 780, its
// products 1,024 with 128 rows).  Few rows: shared memory's 128 bytes a clock, some 80% taken (V
// written 256 clocks and read by the products 256 to 300, the raw tile written and read 300, Q, P,
// scales and factors the rest).  Many rows: the chain of a tile, at half the issue slots, of 3,600 (8
// rows) to 10,300 (128) warp instructions -- conversions and packed multiplies of 32,768 values,
// per score a multiply-add, a power of two, a rounding and a sum.  (Without the powers of two: 2%
// less.)  The registers are all taken: with 64 and 128 rows some 30 bytes a thread are spilled, 70 to 120 with options.
// 128 rows as two tiles of 64: 327 us.  One CTA of sixteen workers up to 64 rows too: 61
// instead of 50 us for 32 sequences, n 4,096, 32 rows.
//
// Split: all pairs' 128-token tiles form one flat range (a pair's start and end count as two
// tiles more), cut equally over the CTAs of a row tile.  A pair that lies in one CTA is
// normalised and written there; others leave (m, l, O) partials that a second kernel joins.
// Tiles wholly before the window of every row are left out.  Every wait is bounded.
#include <algorithm>
#include <cfloat>
#include <mutex>

#include "common.cuh"
#include "flat_plan.cuh"
#include "kernels.h"
#include "quantize.cuh"
#include "tcgen05.cuh"

namespace nvfp4kv {

namespace {

// Up to 64 rows a tile: eight workers, two CTAs an SM.  With 128: sixteen workers, one CTA.
template <int N>
constexpr bool kWide = N == 128;
template <int N>
constexpr int kWorkersT = kWide<N> ? 512 : 256;
template <int N>
constexpr int kThreadsT = kWorkersT<N> + 64;  // + the MMA warp and the load warp
template <int N>
constexpr int kCtasT = kWide<N> ? 1 : 2;      // CTAs an SM
constexpr int kTileT = kTreeTile;             // tokens a tile
constexpr int kBlockT = kTileT * 128;         // bytes of a column block: 64 dims (or rows of P) of 128 tokens
constexpr int kGroupT = 2304;                 // bytes of a 16-token group
constexpr int kRawT = 8 * kGroupT;            // a raw tile
constexpr uint32_t kWaitLimitT = 1u << 24;
constexpr float kNegInfT = -__builtin_huge_valf();
constexpr float kRescaleT = 8.0f;
constexpr float kPOffsetT = 7.0f;             // P = 2^(z - m + 7): at most 2^15
constexpr float kNoMaxT = 3.402823466e38f;    // the offset while every score was -inf
constexpr int kPairUnits = kTreePairUnits;    // what a pair's start and end cost a CTA, in tiles

template <int N>
struct TSmem {
    static constexpr bool kW = kWide<N>;
    static constexpr int kStages = N == 64 ? 2 : 3;
    static constexpr int kQBlock = N * 128;                       // a column block of Q, [N][64]
    static constexpr int kQ = 0;
    static constexpr int kV = 2 * kQBlock;                        // two column blocks
    static constexpr int kP = kV + (kW ? 3 : 1) * 2 * kBlockT;    // FP16 [N / 64][128 tokens][64]
    static constexpr int kRaw = kP + (kW ? 2 : 1) * kBlockT;
    static constexpr int kBar = kRaw + kStages * kRawT;
    static constexpr int kFirstRaw = kW ? 8 : 3;                  // ready done drain; 128 rows: k_ready[2] scored[2] pv_odd too
    static constexpr int kNumBars = kFirstRaw + 2 * kStages;      // raw_full[] raw_free[]
    static constexpr int kMisc = kBar + 8 * kNumBars;             // tmem base, abort, valid[kStages]
    static constexpr int kM = (kMisc + 8 + 4 * kStages + 15) & ~15;   // float m[N], fac[N], alpha[N], off[N], slope[N], depth[N], in[N]
    static constexpr int kRow = kM + 7 * N * 4;                   // int row[N] (-1: none), draft[N]
    static constexpr int kWarpMax = kRow + 2 * N * 4;             // float [warpgroups][4][rows of one]
    static constexpr int kMask = kWarpMax + 4 * N * 4;            // u64 mask[64], int depth[64]
    static constexpr int kNan = kMask + 64 * 12;                  // u32 nan[1 + 64 + 64]: of all rows, of drafts, of the window's edge
    static constexpr int kBytes = kNan + 4 * 129;
    // TMEM columns: O at 0, S (two with 128 rows), K[2]
    static constexpr uint32_t kColS = N, kColK = (kW ? 3 : 2) * N, kCols = kW ? 512 : 256;
    static_assert(kColK + 128 <= kCols && kCtasT<N> * kCols <= 512, "TMEM columns");
    static_assert(kV % 1024 == 0 && kP % 1024 == 0 && kRaw % 1024 == 0 && kBar % 16 == 0 && kMask % 8 == 0, "alignment");
    static_assert(kCtasT<N> * (kBytes + 1024) <= 228 * 1024, "shared memory of an SM");
    static_assert(sizeof(FlatScratch<kThreadsT<N>>) <= 2 * kBlockT, "the plan's scratch lies in the V tile");
};

struct TreeArgs {
    const uint8_t *pool;
    int64_t num_pages, slab;
    int P, log2P, Hkv, G, Hq, B, max_pages, max_q;
    int64_t total_q, cap;
    const uint16_t *q;
    const int32_t *cu_q, *block_table, *seq_lens;
    const uint64_t *mask;
    const float *slopes;      // [Hq] or nullptr
    float score_log2;         // sm_scale * g_K * log2(e)
    float cap_log2;           // cap * log2(e), 0: none
    float cap_in;             // 2 log2(e) / cap * sm_scale * g_K for a cap of kCapFrom to kCapTo, 0 for others
    float cap_rcp;            // 1 / (cap * log2(e))
    int window;               // 0: none
    float gv;
    __nv_bfloat16 *out;
    float2 *part_ml;          // [row tiles][slots][N]
    float *part_acc;          // [row tiles][slots][N][128]
    int splits;
    unsigned *err;
};

// A sequence as the call describes it: d = 0 where that is inconsistent (which is flagged elsewhere).
struct Seq {
    int q0, d, n, base, t0, nt;   // first query row, drafts, tokens, tokens before the drafts, first tile, tiles
};

__device__ __forceinline__ Seq seq_of(const TreeArgs &a, int b) {
    Seq s;
    const int32_t q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
    s.n = clamp_rows(__ldg(a.seq_lens + b), a.cap);
    s.q0 = q0;
    const bool fits = q0 >= 0 && q1 >= q0 && q1 <= a.total_q;
    s.d = fits ? min(q1 - q0, a.max_q) : 0;
    if (s.d > s.n) s.n = 0;       // drafts that the cache does not hold: nothing is seen
    s.base = max(s.n - s.d, 0);
    s.t0 = a.window > 0 && s.base > a.window ? (s.base - a.window) / kTileT : 0;
    s.nt = (s.n + kTileT - 1) / kTileT - s.t0;
    return s;
}

// Units of sequence b's pairs in the flat order of a row tile whose first row is r0.
__device__ __forceinline__ int pair_units(const TreeArgs &a, const Seq &s, int r0) {
    return s.nt > 0 && s.d * a.G > r0 ? s.nt + kPairUnits : 0;
}

// The pairs of a CTA's range in order, and of each its tiles [t, te) that lie in the range.
struct TreeIter {
    int b, kv, t, te;
    Seq s;
    int left;        // units of the range from tile t on
};

__device__ __forceinline__ bool next_pair(const TreeArgs &a, TreeIter &it, int r0) {
    it.left -= it.te - it.t + kPairUnits;
    if (it.left <= 0) return false;
    if (++it.kv == a.Hkv) {
        it.kv = 0;
        do {         // left > 0: a later sequence has tiles
            it.s = seq_of(a, ++it.b);
        } while (pair_units(a, it.s, r0) == 0);
    }
    it.t = 0;
    it.te = min(it.s.nt, it.left);
    return true;
}

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const volatile int *abort_flag) {
    for (uint32_t n = 0; n < kWaitLimitT; n++) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 63) == 63 && *abort_flag) return false;
    }
    return false;
}

// Brings `bytes` (a multiple of 16) at p, 16-byte aligned, to L2.
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two scale bytes of a token and of the token eight behind it (rel: its index, from the base of the drafts on), some
// NaN: those are noted and set to zero.  See s_nan.
__device__ __noinline__ uint32_t without_nan(uint32_t scales, unsigned *s_nan, int rel, int window, int eq) {
    for (int i = 0; i < 4; i++) {
        if (((scales >> (8 * i)) & 0x7fu) != 0x7fu) continue;
        const unsigned bit = 1u << (2 * eq + (i & 1));
        const int at = rel + 8 * (i >> 1), edge = at + window;   // edge: from the window of the first draft on
        if (at >= 0) atomicOr(s_nan + 1 + min(at, 63), bit);
        else if (window <= 0 || edge >= 64) atomicOr(s_nan, bit);
        else if (edge >= 0) atomicOr(s_nan + 65 + edge, bit);
        scales &= ~(0xffu << (8 * i));
    }
    return scales;
}

// cap tanh(x) of e2x = 2 x log2(e).  Each step is off by some 2^-23 of the cap, together 1.3 2^-22 of it: of a score
// up to kCapTo that moves its weight by 2^-14.6 at most.
constexpr double kCapFrom = 0x1p-10, kCapTo = 128.0;

__device__ __forceinline__ float capped(float e2x, float cap) { return fmaf(-2.0f * cap, rcp_approx(ex2(e2x) + 1.0f), cap); }

// z = cap tanh(z / cap) of any cap (rcp: 1 / cap), off by at most 2^-20 of itself.  With x = z / cap: below 1/2, z
// tanh(x) / x by a polynomial in x^2 (off by 2^-26; coefficients solved for the least largest relative error); above,
// capped(), off by 2^-22 of the cap, which is 2.2 z at most there.
__device__ __forceinline__ void any_cap(float (&z)[4], float cap, float rcp) {
    float t[4];
    bool large = false;
#pragma unroll
    for (int c = 0; c < 4; c++) {
        const float x = z[c] * rcp, y = x * x;
        large = large || !(y < 0.25f);
        const float p = fmaf(fmaf(fmaf(0.017135007f, y, -0.052986074f), y, 0.13324779f), y, -0.3333307f);
        t[c] = fmaf(z[c], p * y, z[c]);
    }
    if (large) {
#pragma unroll
        for (int c = 0; c < 4; c++) {
            const float x = z[c] * rcp;
            if (!(x * x < 0.25f)) t[c] = capped(2.8853900817779268f * x, cap);
        }
    }
#pragma unroll
    for (int c = 0; c < 4; c++) z[c] = t[c];
}

__device__ __noinline__ float4 any_cap_called(float4 z, float cap, float rcp) {
    float v[4] = {z.x, z.y, z.z, z.w};
    any_cap(v, cap, rcp);
    return make_float4(v[0], v[1], v[2], v[3]);
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
template <int N>
__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 5, %0;" ::"n"(kWorkersT<N>) : "memory"); }

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
    for (int w = CW / 2; w; w >>= 1) {
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

template <int C>
__device__ __forceinline__ void load_columns(uint32_t taddr, uint32_t (&r)[C]) {
    if constexpr (C == 32) tc_ld32(taddr, r);
    else tc_ld(taddr, r);
}

// OPT: the scores are capped or biased, or their factor is not positive.
template <int N, bool OPT>
__global__ void __launch_bounds__(kThreadsT<N>, kCtasT<N>) tree_kernel(TreeArgs a) {
    using L = TSmem<N>;
    constexpr bool W = kWide<N>;
    constexpr int kWarps = kWorkersT<N> / 32, kMmaWarp = kWarps, kLoadWarp = kWarps + 1;
    constexpr int CW = N / (kWarps / 4);          // rows per warpgroup
    constexpr int S = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBar);
    uint64_t *ready = bars, *done = bars + 1, *drain = bars + 2, *raw_full = bars + L::kFirstRaw, *raw_free = raw_full + S;
    // 128 rows: pairs of barriers, by the tile's parity -- the first waits of a tile may follow the next one's arrivals
    auto k_ready = [&](uint32_t j) { return bars + 3 + (j & 1); };
    auto scored = [&](uint32_t j) { return bars + 5 + (j & 1); };
    auto pv_done = [&](uint32_t j) { return j & 1 ? bars + 7 : done; };
    uint32_t &tmem_base = *reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    volatile int *s_valid = abort_flag + 1;
    float *s_m = reinterpret_cast<float *>(smem + L::kM), *s_fac = s_m + N, *s_alpha = s_fac + N, *s_off = s_alpha + N;
    float *s_slope = s_off + N, *s_dep = s_slope + N, *s_in = s_dep + N;
    int *s_row = reinterpret_cast<int *>(smem + L::kRow), *s_draft = s_row + N;
    uint64_t *s_mask = reinterpret_cast<uint64_t *>(smem + L::kMask);
    int *s_depth = reinterpret_cast<int *>(s_mask + 64);
    // A value block that is NaN would reach every row (0 times NaN is NaN): it is multiplied as zeros, noted here
    // (bit b: block b) and put into the outputs of the rows that see its token.
    unsigned *s_nan = reinterpret_cast<unsigned *>(smem + L::kNan);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r0 = blockIdx.y * N;
    if (tid == 0) {
        for (int i = 0; i < L::kNumBars; i++)
            mbar_init(&bars[i], i == 0 || i >= L::kFirstRaw + S ? kWarps : W && (i == 3 || i == 4) ? kWarps / 2 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (tid < 129) s_nan[tid] = 0;
    pdl_wait();               // everything read or written may belong to earlier work of the stream
    pdl_launch_dependents();
    if (warp == kMmaWarp) tc_alloc(&tmem_base, L::kCols);

    int b0;
    unsigned first, u0 = 0, u1 = 0;
    flat_locate<kThreadsT<N>>(
        *reinterpret_cast<FlatScratch<kThreadsT<N>> *>(smem + L::kV), a.B,
        [&](int b) { return (unsigned)a.Hkv * pair_units(a, seq_of(a, b), r0); },
        [&](unsigned total) {
            const FlatCut cut(total, a.splits);
            u0 = cut.begin(blockIdx.x);
            u1 = cut.begin(blockIdx.x + 1);
            return u0 < u1 ? u0 : kFlatNone;
        },
        b0, first);
    if (warp == kMmaWarp && blockIdx.y == 0) {   // what is out of range, and the rows of sequences without tokens
        for (int b = blockIdx.x; b < a.B; b += a.splits) {
            const Seq s = seq_of(a, b);
            const int32_t n = __ldg(a.seq_lens + b), q1 = __ldg(a.cu_q + b + 1);
            if (lane == 0) {
                if (n < 0 || (int64_t)n > a.cap) flag_error(a.err, kErrSeqLen);
                const bool fits = s.q0 >= 0 && q1 >= s.q0 && q1 <= a.total_q;
                if (!fits || q1 - s.q0 > a.max_q || (n > 0 && s.d > clamp_rows(n, a.cap))) flag_error(a.err, kErrDraft);
            }
            if (s.n > 0 || s.d == 0) continue;
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + (int64_t)s.q0 * a.Hq * kHeadDim);
            for (int i = lane; i < s.d * a.Hq * (kHeadDim / 8); i += 32) dst[i] = make_uint4(0, 0, 0, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    TreeIter it = {};
    it.b = b0;
    if (u0 < u1) {
        it.s = seq_of(a, b0);
        const int per = it.s.nt + kPairUnits, rel = (int)(u0 - first), in = rel % per;
        it.kv = rel / per;
        it.t = max(0, in - kPairUnits);
        it.left = (int)(u1 - u0) - max(0, kPairUnits - in);
        it.te = min(it.s.nt, it.t + it.left);
    }
    if (it.left <= 0) {   // a range without tiles
        if (warp == kMmaWarp) tc_dealloc(tmem_base, L::kCols);
        return;
    }
    const uint32_t tmem = tmem_base, sbase = smem_u32(smem);
    if (warp == kMmaWarp) {
        // ---------------- the MMA warp: the whole warp runs the loop, one elected lane issues
        constexpr uint32_t idesc_s = idesc_f16_f32(128, N, false);
        constexpr uint32_t idesc_o = idesc_a_mn_major(idesc_f16_f32(128, N, true));
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const bool leader = elect_one();
        // operand descriptors; a step adds its byte offset / 16 to the address field
        const uint64_t dQ = smem_desc_sw128(sbase + L::kQ, 16, 1024), dP = smem_desc_sw128(sbase + L::kP, kBlockT, 1024);
        const uint64_t dV = smem_desc_sw128(sbase + L::kV, kBlockT, 1024);
        auto scores = [&](uint32_t kb, uint32_t sb) {      // S^T from K's buffer kb
#pragma unroll
            for (int kk = 0; kk < 8; kk++)
                tc_mma_bf16_tmem_a(tm + L::kColS + sb * N, tm + L::kColK + kb * 64 + kk * 8,
                                   dQ + ((kk >> 2) * (L::kQBlock / 16) + (kk & 3) * 2), idesc_s, kk > 0);
        };
        auto output = [&](uint32_t vb, uint32_t acc) {     // O^T (+)= V^T P^T; 16 tokens: 2,048 bytes of a column block, and of P
            const uint64_t v = dV + vb * (2 * kBlockT / 16);
#pragma unroll
            for (int kk = 0; kk < 8; kk++) tc_mma_bf16(tm, v + kk * 128, dP + kk * 128, idesc_o, kk > 0 ? 1u : acc);
        };
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            const bool good = __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
            tc_fence_after();
            return good;
        };
        bool ok = true;
        if constexpr (W) {
            uint32_t j = 0, kp = 0, vb = 0;                // tile, K tiles taken, V's buffer
            do {
                for (int t = it.t - 1; ok && t < it.te; t++) {   // (t = it.t - 1: the pair's Q and its first K)
                    if (t + 1 < it.te) {
                        ok = wait(k_ready(kp), (kp >> 1) & 1);
                        if (!ok) break;
                        if (leader) {
                            scores(kp & 1, kp & 1);
                            tc_commit(scored(kp));
                        }
                        kp++;
                    }
                    if (t < it.t) continue;
                    ok = wait(ready, j & 1);
                    if (!ok) break;
                    if (leader) {
                        output(vb, t == it.t ? 0u : 1u);
                        tc_commit(pv_done(j));
                    }
                    vb = vb == 2 ? 0 : vb + 1;
                    j++;
                }
            } while (ok && next_pair(a, it, r0));
        } else {
            uint32_t phase = 0, kb = 0;                    // kb: K's buffer
            do {
                for (int t = it.t - 1; t < it.te; t++) {   // (t = it.t - 1: the pair's Q and its first K)
                    ok = wait(ready, phase++ & 1);
                    if (!ok) break;
                    if (leader) {
                        if (t + 1 < it.te) scores(kb, 0);  // of the next tile
                        if (t >= it.t) output(0, t == it.t ? 0u : 1u);
                        tc_commit(done);
                    }
                    if (t + 1 < it.te) kb ^= 1u;
                }
            } while (ok && next_pair(a, it, r0));
        }
        if (!ok && leader) {
            if (!*abort_flag) flag_error(a.err, kErrTimeout);
            *abort_flag = 1;
            tc_commit(drain);   // no product may still read the CTA's memory when it ends
            mbar_wait_bounded(drain, 0, kWaitLimitT, nullptr);
        }
        __syncwarp();
    } else if (warp == kLoadWarp) {
        // ---------------- the load warp: lane g < 8 copies group g of each tile
        uint32_t j = 0, st = 0, ph = 0;
        bool ok = true;
        do {
            const int32_t *table = a.block_table + (int64_t)it.b * a.max_pages;
            const uint8_t *pool = a.pool + it.kv * a.slab;
            int tok = (it.s.t0 + it.t) * kTileT + 16 * lane;
            auto page_at = [&](int x) { return lane < 8 && x < it.s.n ? __ldg(table + (x >> a.log2P)) : -1; };
            int32_t page = page_at(tok);
            for (int t = it.t; t < it.te; t++, j++, tok += kTileT) {
                const int32_t next = t + 1 < it.te ? page_at(tok + kTileT) : -1;
                if (j >= S) ok = __all_sync(0xffffffffu, wait_bar(&raw_free[st], ph ^ 1u, abort_flag));
                if (!ok) break;
                const bool want = lane < 8 && tok < it.s.n, good = want && page >= 0 && page < a.num_pages;
                if (want && !good) flag_error(a.err, kErrPage);
                const unsigned mask = __ballot_sync(0xffffffffu, good);
                if (lane == 0) {
                    s_valid[st] = (int)mask;
                    mbar_arrive_expect_tx(&raw_full[st], (uint32_t)__popc(mask) * kGroupT);
                }
                __syncwarp();
                auto group_at = [&](int32_t pg, int x) {
                    return pool + (int64_t)pg * a.Hkv * a.slab + ((x & (a.P - 1)) >> 4) * kGroupT;
                };
                if (good) bulk_g2s(smem + L::kRaw + st * kRawT + lane * kGroupT, group_at(page, tok), kGroupT, &raw_full[st]);
                // With two stages the tile after it comes to L2 while its place in the ring is still in use (64 rows: 188
                // us without, 183 so; with three stages nothing).
                if (N == 64 && next >= 0 && next < a.num_pages) prefetch_l2(group_at(next, tok + kTileT), kGroupT);
                page = next;
                if (++st == S) st = 0, ph ^= 1u;
            }
        } while (ok && next_pair(a, it, r0));
        if (!ok) {
            if (lane == 0 && !*abort_flag) flag_error(a.err, kErrTimeout);
            *abort_flag = 1;
        }
        // no copy may still be writing when the CTA ends
        for (uint32_t i = j > S ? j - S : 0; i < j; i++)
            mbar_wait_bounded(&raw_full[i % S], (i / S) & 1, kWaitLimitT, nullptr);
    } else {
        // ---------------- expanding and softmax
        // A wait that gave up sets the abort flag, which ends every other wait; the warps then
        // still run through their tiles (on meaningless values), so that no barrier is left
        // short of a warp.
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!wait_bar(bar, parity, abort_flag) && !*abort_flag) {
                *abort_flag = 1;
                flag_error(a.err, kErrTimeout);
            }
            __syncwarp();
        };
        const int wg = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;   // softmax: rows' part, token
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const int er = lane >> 2, eq = lane & 3;
        // expanding: 16-token group grp of the tile (its TMEM lanes are this warp's to reach)
        const int grp = 2 * quarter + (wg & 1);
        uint32_t ks = 0, ksp = 0, vs = 0, kb = 0;   // the raw stages whose K and V come next, K's parity and buffer

        // 16 dims a word pair of 16-byte piece eq, times the scales of its two blocks
        auto scaled = [&](const uint32_t (&w)[4], uint32_t s0, uint32_t s1, uint32_t (&f)[16]) {
#pragma unroll
            for (int m = 0; m < 4; m++) {
                e2m1x8_to_f16x2x4(w[m], f[4 * m], f[4 * m + 1], f[4 * m + 2], f[4 * m + 3]);
#pragma unroll
                for (int i = 0; i < 4; i++) f[4 * m + i] = hmul2(f[4 * m + i], m < 2 ? s0 : s1);
            }
        };
        auto free_stage = [&](uint32_t st) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_free[st]);
        };
        // K of the next raw tile to TMEM; returns the groups that the tile holds.  (Rows that do
        // not exist: their scores are masked.)
        auto expand_k = [&]() {
            wait(&raw_full[ks], ksp);
            const int held = s_valid[ks];
            const uint8_t *g = smem + L::kRaw + ks * kRawT + grp * kGroupT;
            uint32_t f[2][16];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int r = er + 8 * e;
                const uint4 c = *reinterpret_cast<const uint4 *>(g + r * 64 + eq * 16);
                const uint32_t s = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(g + 1024 + r * 8 + eq * 2));
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
                scaled(w, __byte_perm(s, 0, 0x1010), __byte_perm(s, 0, 0x3232), f[e]);
            }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t v[16] = {f[0][8 * h], f[0][8 * h + 1], f[1][8 * h], f[1][8 * h + 1],
                                        f[0][8 * h + 2], f[0][8 * h + 3], f[1][8 * h + 2], f[1][8 * h + 3],
                                        f[0][8 * h + 4], f[0][8 * h + 5], f[1][8 * h + 4], f[1][8 * h + 5],
                                        f[0][8 * h + 6], f[0][8 * h + 7], f[1][8 * h + 6], f[1][8 * h + 7]};
                tc_st_16x256_x4(tmem + ((uint32_t)(16 * grp) << 16) + L::kColK + 64 * kb + 32 * h, v);
            }
            kb ^= 1u;
            if (W) free_stage(ks);
            if (++ks == S) ks = 0, ksp ^= 1u;
            return held;
        };
        // V of the tile of stage vs to shared memory, buffer vb; rows: those of the group that exist.
        // Lanes q >= 2 take rows r ^ 2, so that a quarter warp's stores meet all banks.
        auto expand_v = [&](int rows, uint32_t vb, const Seq &sq) {
            const int r0v = er ^ (eq & 2);
            const uint8_t *g = smem + L::kRaw + vs * kRawT + grp * kGroupT + 1152;
            uint8_t *blk = smem + L::kV + (2 * vb + (eq >> 1)) * kBlockT + (16 * grp + r0v) * 128;
            const uint8_t *gs = g + 1024 + 2 * eq * 16 + r0v;
            uint32_t scales = gs[0] | (uint32_t)gs[16] << 8 | (uint32_t)gs[8] << 16 | (uint32_t)gs[24] << 24;   // of rows r0v, r0v + 8
            if (rows < 16) {                              // rows that do not exist may hold anything: zeros
                if (r0v >= rows) scales &= 0xffff0000u;
                if (r0v + 8 >= rows) scales &= 0x0000ffffu;
            }
            if (((scales & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u)
                scales = without_nan(scales, s_nan, sq.n - rows + r0v - sq.base, a.window, eq);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int r = r0v + 8 * e;
                uint4 c = *reinterpret_cast<const uint4 *>(g + r * 64 + eq * 16);
                uint32_t s = scales >> (16 * e);
                s = e4m3x2_to_f16x2(s);
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
                uint32_t f[16];
                scaled(w, __byte_perm(s, 0, 0x1010), __byte_perm(s, 0, 0x3232), f);
#pragma unroll
                for (int m = 0; m < 4; m++)
                    *reinterpret_cast<uint4 *>(blk + e * 1024 + ((((eq & 1) * 4 + m) ^ (r0v & 7)) << 4)) =
                        make_uint4(f[4 * m], f[4 * m + 1], f[4 * m + 2], f[4 * m + 3]);
            }
            free_stage(vs);
            if (++vs == S) vs = 0;
        };
        // 128 rows: K by the first two warpgroups, V by the others, of tile j (from tok0 on).  V's buffer was read last by
        // the product of tile j - 3 (which is done where the tile is its pair's first).
        uint32_t vb = 0;
        auto report_k = [&](uint32_t j) {
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(k_ready(j));
        };
        auto expand_wide = [&](const Seq &sq, int tok0, uint32_t j, bool first) {
            if (wg < 2) {
                const int held = expand_k();
                if (!first) report_k(j);
                return held;
            }
            wait(&raw_full[vs], ksp);
            const int held = s_valid[vs];
            if (!first && j >= 3) wait(pv_done(j - 3), ((j - 3) >> 1) & 1);
            expand_v((held >> grp) & 1 ? sq.n - (tok0 + 16 * grp) : 0, vb, sq);
            vb = vb == 2 ? 0 : vb + 1;
            if (vs == 0) ksp ^= 1u;
            return held;
        };
        // What this warp has put into TMEM and shared memory is the MMA warp's.
        auto hand_over = [&]() {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ready);
        };
        // A pair's Q, the rows' factors and the tree: requested before the pair's first tile is expanded, laid out
        // after it.  (The previous pair's products and its epilogue are done.)
        uint2 qw[N / kWarps];
        int at[N / kWarps];                     // a row of q, -1: none
        uint64_t tree = 0;
        auto fetch_pair = [&](const TreeIter &x) {
            const int rows = x.s.d * a.G;
#pragma unroll
            for (int k = 0; k < N / kWarps; k++) {
                const int r = r0 + warp + kWarps * k, i = r / a.G;
                at[k] = r < rows ? (x.s.q0 + i) * a.Hq + x.kv * a.G + (r - i * a.G) : -1;
                qw[k] = make_uint2(0, 0);
                if (r < rows) qw[k] = __ldg(reinterpret_cast<const uint2 *>(a.q + (int64_t)at[k] * kHeadDim) + lane);
            }
            tree = 0;
            if (tid < x.s.d) {
                const uint64_t all = x.s.d >= 64 ? ~0ull : (1ull << x.s.d) - 1;
                tree = (a.mask ? __ldg(reinterpret_cast<const unsigned long long *>(a.mask) + x.s.q0 + tid) : (2ull << tid) - 1) & all;
            }
        };
        auto store_pair = [&]() {
            constexpr int R = N / kWarps;       // rows a warp: their scalars are lanes 0 .. R - 1's
            int my_kq = 0, my_at = -1;
            uint32_t m[R];
#pragma unroll
            for (int k = 0; k < R; k++) {
                const uint32_t x = max_u16x2(qw[k].x & 0x7fff7fffu, qw[k].y & 0x7fff7fffu);
                m[k] = __reduce_max_sync(0xffffffffu, max(x >> 16, x & 0xffffu));
            }
#pragma unroll
            for (int k = 0; k < R; k++) {
                const int c = warp + kWarps * k;
                const uint2 w = qw[k];
                // 2^kq puts the row's largest value into [2^14, 2^15)
                const int kq = m[k] ? min(126, max(-126, 14 - ((int)(m[k] >> 7) - 127))) : 0;
                const float sc = __uint_as_float((uint32_t)(kq + 127) << 23);
                // dims 4 lane .. + 3 = 32 q + 4 a + e lie at position 16 a + 4 q + e
                const int pos = 16 * (lane & 7) + 4 * (lane >> 3);
                *reinterpret_cast<uint2 *>(smem + L::kQ + (pos >> 6) * L::kQBlock + sw128_off(c, (pos & 63) >> 3) + (pos & 7) * 2) =
                    make_uint2(f32x2_to_f16x2(bf16_hi(w.x) * sc, bf16_lo(w.x) * sc),
                               f32x2_to_f16x2(bf16_hi(w.y) * sc, bf16_lo(w.y) * sc));
                if (lane == k) my_kq = kq, my_at = at[k];
            }
            if (lane < R) {
                const int c = warp + kWarps * lane;
                const float fac = (OPT && a.cap_in != 0.f ? a.cap_in : a.score_log2) * __uint_as_float((uint32_t)(127 - my_kq) << 23);
                // (a positive factor stays one, so that minus infinity times it is minus infinity: no score
                // reaches 2^34, and 2^-92 is none)
                s_fac[c] = OPT ? 1.f : fmaxf(fac, 0x1p-126f);
                if (OPT) s_in[c] = fac;
                s_m[c] = kNegInfT;
                s_off[c] = kNoMaxT;
                s_row[c] = my_at;
                s_draft[c] = min((r0 + c) / a.G, 63);
                if (OPT) s_slope[c] = a.slopes && my_at >= 0 ? __ldg(a.slopes + my_at % a.Hq) * 1.4426950408889634f : 0.f;
            }
            if (tid < 64) {
                s_mask[tid] = tree;
                s_depth[tid] = __popcll(tree) - 1;
            }
            if (W) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // Q, before any warp reports K
            workers_sync<N>();
            if (OPT) {
                if (tid < N) s_dep[tid] = (float)s_depth[s_draft[tid]];
                workers_sync<N>();
            }
        };
        // Which of the warpgroup's rows do not see the thread's token (bit c: row c).
        auto unseen = [&](const Seq &s, int tok, int held) {
            const int rel = tok - s.base, jj = rel < 0 ? 0 : min(rel, 63), key = rel < 0 ? rel : s_depth[jj];
            const bool there = tok < s.n && ((held >> (row >> 4)) & 1);
            uint32_t gone = 0;
#pragma unroll 1
            for (int c = 0; c < CW; c++) {
                const int i = s_draft[wg * CW + c];
                const bool sees = there && (rel < 0 || (s_mask[i] >> jj) & 1) && (a.window <= 0 || key > s_depth[i] - a.window);
                gone |= sees ? 0u : 1u << c;
            }
            return gone;
        };

        uint32_t phase = 0;                         // up to 64 rows: products awaited; 128: tiles
        do {
            fetch_pair(it);
            int tok0 = (it.s.t0 + it.t) * kTileT;
            int held = 0, held_next;                // the groups that a raw tile holds
            if constexpr (W) {
                held_next = expand_wide(it.s, tok0, phase, true);
                store_pair();
                if (wg < 2) report_k(phase);
            } else {
                held_next = expand_k();
                store_pair();
                hand_over();
            }
            float l[CW];
#pragma unroll
            for (int c = 0; c < CW; c++) l[c] = 0.f;
            for (int t = it.t; t < it.te; t++, tok0 += kTileT) {
                held = held_next;
                if constexpr (W) {
                    if (t + 1 < it.te) held_next = expand_wide(it.s, tok0 + kTileT, phase + 1, false);
                    wait(scored(phase), (phase >> 1) & 1);
                    tc_fence_after();
                } else {
                    // The products handed over last run while K of the next tile is unpacked.
                    if (t + 1 < it.te) held_next = expand_k();
                    // This tile's scores are there, O^T holds the tiles before: V and P may be written.
                    wait(done, phase++ & 1);
                    tc_fence_after();
                    expand_v((held >> grp) & 1 ? it.s.n - (tok0 + 16 * grp) : 0, 0, it.s);
                }

                // ---- softmax of the token's scores for the warpgroup's rows
                const int tok = tok0 + row;
                // edge: a token of the tile that some row does not see
                const bool edge = tok0 + kTileT > it.s.base || (a.window > 0 && tok0 <= it.s.n - 1 - a.window) || held != 0xff;
                const uint32_t tS = tmem + lanes + L::kColS + (W ? (phase & 1) * N : 0) + wg * CW, tO = tmem + lanes + wg * CW;
                if (OPT || edge) {                  // in place: the capped and biased scores, minus infinity where nothing is seen
                    const uint32_t gone = edge ? unseen(it.s, tok, held) : 0u;
                    const int rel = tok - it.s.base;
                    const float key = OPT ? (float)(rel < 0 ? rel : s_depth[min(rel, 63)]) : 0.f;   // the token's position, from base on
#pragma unroll 1
                    for (int c0 = 0; c0 < CW; c0 += 8) {
                        uint32_t x[8];
                        tc_ld8(tS + c0, x);
                        tc_wait_ld();
                        if (OPT) {
                            float in[8], slope[8], dep[8];
#pragma unroll
                            for (int i = 0; i < 2; i++) {
                                *reinterpret_cast<float4 *>(in + 4 * i) = reinterpret_cast<const float4 *>(s_in + wg * CW + c0)[i];
                                *reinterpret_cast<float4 *>(slope + 4 * i) = reinterpret_cast<const float4 *>(s_slope + wg * CW + c0)[i];
                                *reinterpret_cast<float4 *>(dep + 4 * i) = reinterpret_cast<const float4 *>(s_dep + wg * CW + c0)[i];
                            }
#pragma unroll
                            for (int c = 0; c < 8; c++) in[c] *= __uint_as_float(x[c]);
                            if (a.cap_in != 0.f) {
#pragma unroll
                                for (int c = 0; c < 8; c++) in[c] = capped(in[c], a.cap_log2);
                            } else if (a.cap_log2 > 0.f) {   // (in line up to 64 rows it costs the other caps registers:
                                // 32 sequences of n 4,096, 32 rows, 68 us instead of 66; called with 128, 16 of n 32,768
                                // take 477 us instead of 457)
#pragma unroll
                                for (int i = 0; i < 2; i++) {
                                    float (&v)[4] = reinterpret_cast<float (&)[4]>(in[4 * i]);
                                    if (W) {
                                        any_cap(v, a.cap_log2, a.cap_rcp);
                                    } else {
                                        const float4 t = any_cap_called(make_float4(v[0], v[1], v[2], v[3]), a.cap_log2, a.cap_rcp);
                                        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
                                    }
                                }
                            }
#pragma unroll
                            for (int c = 0; c < 8; c++) x[c] = __float_as_uint(fmaf(slope[c], key - dep[c], in[c]));
                        }
#pragma unroll
                        for (int c = 0; c < 8; c++)
                            if ((gone >> (c0 + c)) & 1) x[c] = 0xff800000u;
                        tc_st8(tS + c0, x);
                    }
                    tc_wait_st();
                }
                // P = 2^d, d = z - m + 7, CH rows at a time.  Up to 64 rows by the maxima as they stand, and again where
                // one has to move; with 128 rows, whose warps have fewer registers to spare, P is formed after the
                // vote from the scores in TMEM (64 rows: 176 us so, 183 after the vote; 128 rows, 8 sequences of up to 2,000:
                // 44 us before, 40 after).
                constexpr int CH = CW < 16 ? CW : 16;
                uint32_t pw[W ? CH / 2 : CW / 2];
                float top, top2;
                auto scan = [&](int c0, auto use) {     // use(c, d of rows c .. c + 3)
                    uint32_t x[CH];
                    load_columns<CH>(tS + c0, x);
                    const float4 *fac = reinterpret_cast<const float4 *>(s_fac + wg * CW + c0);
                    const float4 *off = reinterpret_cast<const float4 *>(s_off + wg * CW + c0);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < CH; i += 4) {
                        const float4 o = off[i / 4], f = fac[i / 4];
                        use(i, fmaf(__uint_as_float(x[i]), f.x, o.x), fmaf(__uint_as_float(x[i + 1]), f.y, o.y),
                            fmaf(__uint_as_float(x[i + 2]), f.z, o.z), fmaf(__uint_as_float(x[i + 3]), f.w, o.w));
                    }
                };
                auto form = [&]() {
                    top = top2 = kNegInfT;
#pragma unroll
                    for (int c0 = 0; c0 < CW; c0 += CH)
                        scan(c0, [&](int i, float d0, float d1, float d2, float d3) {
                            top = max3(top, d0, d1);
                            top2 = max3(top2, d2, d3);
                            if (!W) {
                                pw[(c0 + i) / 2] = f32x2_to_f16x2(ex2(d1), ex2(d0));
                                pw[(c0 + i) / 2 + 1] = f32x2_to_f16x2(ex2(d3), ex2(d2));
                            }
                        });
                };
                bool moves = t == it.t;             // (a pair's first tile sets them)
                if (!moves) {
                    form();
                    moves = group_any(wg, fmaxf(top, top2) > kRescaleT + kPOffsetT);
                }
                if (moves) {
                    float *wmax = reinterpret_cast<float *>(smem + L::kWarpMax) + wg * 4 * CW;
                    int mine = 0;
#pragma unroll 1
                    for (int c0 = 0; c0 < CW; c0 += 8) {
                        uint32_t x[8];
                        tc_ld8(tS + c0, x);
                        tc_wait_ld();
#pragma unroll
                        for (int c = 0; c < 8; c++) {
                            const int mx = __reduce_max_sync(0xffffffffu, ordered(__uint_as_float(x[c]) * s_fac[wg * CW + c0 + c]));
                            if (lane == c0 + c) mine = mx;
                        }
                    }
                    if (lane < CW) wmax[quarter * CW + lane] = unordered(mine);
                    group_sync(wg);
                    if (quarter == 0 && lane < CW) {
                        const float mx = fmaxf(fmaxf(wmax[lane], wmax[CW + lane]), fmaxf(wmax[2 * CW + lane], wmax[3 * CW + lane]));
                        const float mo = s_m[wg * CW + lane], mn = fmaxf(mo, mx);
                        s_alpha[wg * CW + lane] = mo == kNegInfT ? 0.f : ex2(mo - mn);
                        s_m[wg * CW + lane] = mn;
                        s_off[wg * CW + lane] = mn == kNegInfT ? kNoMaxT : kPOffsetT - mn;
                    }
                    group_sync(wg);
#pragma unroll
                    for (int c = 0; c < CW; c++) l[c] *= s_alpha[wg * CW + c];
                    if (t > it.t) {                 // O^T holds the earlier tiles: rescale the warpgroup's rows
                        if (W) {
                            wait(pv_done(phase - 1), ((phase - 1) >> 1) & 1);
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int c0 = 0; c0 < CW; c0 += 8) {
                            uint32_t x[8];
                            tc_ld8(tO + c0, x);
                            tc_wait_ld();
#pragma unroll
                            for (int c = 0; c < 8; c++)
                                x[c] = __float_as_uint(__uint_as_float(x[c]) * s_alpha[wg * CW + c0 + c]);
                            tc_st8(tO + c0, x);
                        }
                        tc_wait_st();
                    }
                    if (!W) form();
                }
                if (W && phase > 0) wait(pv_done(phase - 1), ((phase - 1) >> 1) & 1);    // P is read
                uint8_t *pt = smem + L::kP + (wg * CW / 64) * kBlockT;
#pragma unroll
                for (int c0 = 0; c0 < CW; c0 += 8) {
                    if (W && c0 % CH == 0)
                        scan(c0, [&](int i, float d0, float d1, float d2, float d3) {
                            pw[i / 2] = f32x2_to_f16x2(ex2(d1), ex2(d0));
                            pw[i / 2 + 1] = f32x2_to_f16x2(ex2(d3), ex2(d2));
                        });
                    const uint32_t *w = pw + (W ? c0 % CH : c0) / 2;
#pragma unroll
                    for (int e = 0; e < 4; e++) add_f16x2(l[c0 + 2 * e], l[c0 + 2 * e + 1], w[e]);
                    *reinterpret_cast<uint4 *>(pt + sw128_off(row, ((wg * CW + c0) & 63) / 8)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                hand_over();
                if (W) phase++;
            }

            // ---- the pair's last tile of this range: normalise, or leave the partial
            if (W) wait(pv_done(phase - 1), ((phase - 1) >> 1) & 1);
            else wait(done, phase++ & 1);
            tc_fence_after();
            float *wsum = reinterpret_cast<float *>(smem + L::kWarpMax) + wg * 4 * CW;
            const float s = column_sums<CW>(l, lane);
            if (lane < CW) wsum[quarter * CW + lane] = s;
            group_sync(wg);
            const bool whole = it.t == 0 && it.te == it.s.nt;
            const int64_t slot = (int64_t)blockIdx.y * ((int64_t)a.splits + (int64_t)a.B * a.Hkv) + blockIdx.x +
                                 (int64_t)it.b * a.Hkv + it.kv;
            if (quarter == 0 && lane < CW) {
                const float m = s_m[wg * CW + lane];
                const float t = (wsum[lane] + wsum[CW + lane]) + (wsum[2 * CW + lane] + wsum[3 * CW + lane]);
                if (!whole) a.part_ml[slot * N + wg * CW + lane] = make_float2(m == kNegInfT ? m : m - kPOffsetT, t);
                s_alpha[wg * CW + lane] = t == 0.f ? 0.f : a.gv / t;      // (a row that sees nothing: zeros)
            }
            workers_sync<N>();
            // NaN blocks: rows' bits into s_draft (which the pair needs no more)
            bool any_nan = false;
            for (int i = lane; i < 129; i += 32) any_nan = any_nan || s_nan[i] != 0;
            any_nan = __any_sync(0xffffffffu, any_nan);
            if (any_nan) {
                unsigned bits = 0;
                if (tid < N) {
                    const int i = s_draft[tid];
                    bits = s_nan[0];
                    for (int x = 0; x < 64; x++) {
                        if ((s_mask[i] >> x & 1) && (a.window <= 0 || s_depth[x] > s_depth[i] - a.window)) bits |= s_nan[1 + x];
                        if (x > s_depth[i]) bits |= s_nan[65 + x];
                    }
                }
                workers_sync<N>();
                if (tid < N) s_draft[tid] = (int)bits;
                if (tid < 129) s_nan[tid] = 0;
                workers_sync<N>();
            }
            float *dst = a.part_acc + (slot * N + wg * CW) * kHeadDim + row;
#pragma unroll 1
            for (int c0 = 0; c0 < CW; c0 += 8) {
                uint32_t x[8];
                tc_ld8(tmem + lanes + wg * CW + c0, x);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; c++) {
                    const int at = s_row[wg * CW + c0 + c];
                    if (at < 0) continue;
                    if (any_nan && (s_draft[wg * CW + c0 + c] >> (row >> 4) & 1)) x[c] = 0x7fc00000u;
                    if (whole)
                        a.out[(int64_t)at * kHeadDim + row] = __float2bfloat16_rn(__uint_as_float(x[c]) * s_alpha[wg * CW + c0 + c]);
                    else
                        dst[(c0 + c) * kHeadDim] = __uint_as_float(x[c]);
                }
            }
            tc_fence_before();
            workers_sync<N>();   // sums, maxima and rows are read: the next pair may write them
        } while (next_pair(a, it, r0));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tc_dealloc(tmem, L::kCols);
}

// Joins the partials of the pairs that several CTAs covered: one warp per row, a float4 a lane.
constexpr int kJoinWarps = 8;

template <int N>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(TreeArgs a) {
    __shared__ unsigned s_sum[2][kJoinWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.z, kv = blockIdx.y, r = blockIdx.x * kJoinWarps + warp;   // (kJoinWarps rows lie in one row tile)
    const int y = blockIdx.x * kJoinWarps / N, r0 = y * N;
    // (the plan's inputs may be read before the wait: the first kernel lets this one start only
    // after its own wait for everything before it, and does not write them)
    const Seq s = seq_of(a, b);
    unsigned before = 0, all = 0;
    for (int x = tid; x < a.B; x += blockDim.x) {
        const unsigned n = (unsigned)a.Hkv * pair_units(a, seq_of(a, x), r0);
        all += n;
        if (x < b) before += n;
    }
    all = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) {
        s_sum[0][warp] = all;
        s_sum[1][warp] = before;
    }
    __syncthreads();
    all = before = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; w++) {
        all += s_sum[0][w];
        before += s_sum[1][w];
    }
    pdl_wait();
    pdl_launch_dependents();
    const int units = pair_units(a, s, r0);
    if (units == 0 || r >= s.d * a.G) return;
    const FlatCut cut(all, a.splits);
    const unsigned start = before + (unsigned)kv * units;
    const int c0 = (int)cut.piece(start + kPairUnits), c1 = (int)cut.piece(start + units - 1);
    if (c0 == c1) return;   // written by its CTA
    const int64_t slot0 = (int64_t)y * ((int64_t)a.splits + (int64_t)a.B * a.Hkv) + (int64_t)b * a.Hkv + kv;
    float m = kNegInfT, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 4;
    for (int c = c0; c <= c1; c += U) {
        float2 ml[U];
        float4 v[U];
#pragma unroll
        for (int k = 0; k < U; k++) {
            ml[k] = make_float2(kNegInfT, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + k <= c1) {
                const int64_t at = (slot0 + c + k) * N + (r - r0);
                ml[k] = __ldcg(a.part_ml + at);
                v[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_acc + at * kHeadDim) + lane);
            }
        }
        float mx = m;
#pragma unroll
        for (int k = 0; k < U; k++) mx = fmaxf(mx, ml[k].x);
        const float f0 = m == kNegInfT ? 0.f : ex2(m - mx);
        l *= f0;
        acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
        for (int k = 0; k < U; k++) {
            if (ml[k].x == kNegInfT && ml[k].y == 0.f) continue;      // it saw nothing
            const float f = ml[k].x == kNegInfT ? ml[k].y : ex2(ml[k].x - mx);   // (no maximum, but a sum: NaN)
            l = fmaf(f, ml[k].y, l);
            acc.x = fmaf(f, v[k].x, acc.x);
            acc.y = fmaf(f, v[k].y, acc.y);
            acc.z = fmaf(f, v[k].z, acc.z);
            acc.w = fmaf(f, v[k].w, acc.w);
        }
        m = mx;
    }
    const float inv = l == 0.f ? 0.f : a.gv / l;
    const int i = r / a.G;
    reinterpret_cast<uint2 *>(a.out + ((int64_t)(s.q0 + i) * a.Hq + kv * a.G + (r - i * a.G)) * kHeadDim)[lane] =
        make_uint2(f32x2_to_bf16x2(acc.y * inv, acc.x * inv), f32x2_to_bf16x2(acc.w * inv, acc.z * inv));
}

struct TreeFns {
    const void *tree[2], *join;
    int smem, threads;
};

template <int N>
TreeFns fns_of() {
    return {{reinterpret_cast<const void *>(&tree_kernel<N, false>), reinterpret_cast<const void *>(&tree_kernel<N, true>)},
            reinterpret_cast<const void *>(&tree_join_kernel<N>), TSmem<N>::kBytes, kThreadsT<N>};
}

// Rows of a CTA's tile.
int tile_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

TreeFns tree_fns(int n) { return n == 16 ? fns_of<16>() : n == 32 ? fns_of<32>() : n == 64 ? fns_of<64>() : fns_of<128>(); }

constexpr int kMaxDevicesT = 64;
std::mutex g_mu_t;
bool g_attr_t[kMaxDevicesT][4][2];
int g_sms_t[kMaxDevicesT];

size_t align256t(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

int tree_auto_splits(int64_t rows, cudaError_t *status) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevicesT)) e = cudaErrorInvalidDevice;
    int sms = 0;
    if (e == cudaSuccess) {
        std::lock_guard<std::mutex> lock(g_mu_t);
        if (!g_sms_t[dev]) e = cudaDeviceGetAttribute(&g_sms_t[dev], cudaDevAttrMultiProcessorCount, dev);
        sms = g_sms_t[dev];
    }
    if (status) *status = e;
    if (e != cudaSuccess) return 0;
    const int64_t n = tile_rows(rows), tiles = (rows + n - 1) / n;
    const int64_t ctas = (n == 128 ? kCtasT<128> : kCtasT<64>) * (int64_t)sms / tiles;
    return ctas > 0 ? (int)ctas : 1;
}

// Workspace: (m, l) partials | their O, one per row tile and (CTA of it, pair) that can meet
size_t tree_workspace_bytes(int batch, int num_kv_heads, int64_t rows, int splits) {
    const size_t n = tile_rows(rows), tiles = (rows + n - 1) / n, slots = (size_t)splits + (size_t)batch * num_kv_heads;
    return align256t(tiles * slots * n * sizeof(float2)) + tiles * slots * n * kHeadDim * sizeof(float);
}

cudaError_t launch_tree(const nvfp4kv_cache &c, const void *q, const int32_t *cu_q, int64_t total_q, int batch,
                        int max_q_len, int num_q_heads, const uint64_t *mask, const int32_t *block_table, int max_pages,
                        const int32_t *seq_lens, float sm_scale, float softcap, int window, const float *slopes,
                        void *out, void *workspace, int splits, unsigned *err, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevicesT)) e = cudaErrorInvalidDevice;
    if (e != cudaSuccess) return e;
    TreeArgs a = {};
    a.pool = static_cast<const uint8_t *>(c.pool);
    a.num_pages = c.num_pages;
    a.slab = (int64_t)144 * c.page_size;
    a.P = c.page_size;
    a.log2P = __builtin_ctz((unsigned)c.page_size);
    a.Hkv = c.num_kv_heads;
    a.Hq = num_q_heads;
    a.G = num_q_heads / c.num_kv_heads;
    a.B = batch;
    a.max_pages = max_pages;
    a.max_q = max_q_len;
    a.total_q = total_q;
    a.cap = (int64_t)max_pages * c.page_size;
    a.q = static_cast<const uint16_t *>(q);
    a.cu_q = cu_q;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.mask = mask;
    a.slopes = slopes;
    const double scale = (double)sm_scale * c.k_global_scale, log2e = 1.4426950408889634;
    a.score_log2 = (float)(scale * log2e);
    // (in FP32's range whatever the cap: a very large one is none, a very small one leaves nothing of the scores)
    a.cap_log2 = (float)std::min(softcap * log2e, (double)FLT_MAX);
    a.cap_rcp = softcap > 0.f ? (float)std::min(1.0 / (softcap * log2e), (double)FLT_MAX) : 0.f;
    a.cap_in = softcap >= kCapFrom && softcap <= kCapTo ? (float)(2.0 * log2e * scale / softcap) : 0.f;
    a.window = window;
    a.gv = c.v_global_scale;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.err = err;
    const int64_t rows = (int64_t)max_q_len * a.G;
    const int n = tile_rows(rows), tiles = (int)((rows + n - 1) / n);
    // The workspace is laid out for the splits that it was sized for.
    const size_t slots = (size_t)splits + (size_t)batch * a.Hkv;
    a.part_ml = static_cast<float2 *>(workspace);
    a.part_acc = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + align256t(tiles * slots * n * sizeof(float2)));
    // No more CTAs than there can be token tiles (by the table's width: the lengths are on the device).
    const int64_t most = (int64_t)batch * a.Hkv * ((a.cap + kTileT - 1) / kTileT);
    a.splits = splits > most ? (int)most : splits;
    const TreeFns f = tree_fns(n);
    const bool opt = softcap > 0.f || slopes || !(a.score_log2 > 0.f);
    {
        std::lock_guard<std::mutex> lock(g_mu_t);
        bool &set = g_attr_t[dev][n == 16 ? 0 : n == 32 ? 1 : n == 64 ? 2 : 3][opt];
        if (!set) {
            e = cudaFuncSetAttribute(f.tree[opt], cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem);
            if (e != cudaSuccess) return e;
            set = true;
        }
    }
    void *args[] = {&a};
    e = launch_pdl(f.tree[opt], dim3((unsigned)a.splits, (unsigned)tiles), (unsigned)f.threads, (size_t)f.smem, stream, args);
    if (e != cudaSuccess || a.splits == 1 || a.cap <= kTileT) return e;   // no pair can have been split
    return launch_pdl(f.join, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps), (unsigned)a.Hkv, (unsigned)batch),
                      32 * kJoinWarps, 0, stream, args);
}

}  // namespace nvfp4kv
