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
// One CTA per SM, 18 warps:
//   * sixteen workers expand a tile and run its softmax.  Expanding: one warp per 16-token
//     group and operand; lane (r, q) holds the q-th 16 bytes of rows r and r + 8.  K goes to
//     TMEM (the store takes a quad's registers as four columns each, so the dims lie there in
//     another order: position 16 a + 4 q + e holds dim 32 q + 4 a + e, and Q's with them), V
//     to a swizzled tile in shared memory.  Softmax: one token (= TMEM lane) a thread, the four
//     warpgroups taking a quarter of the rows each; a lazily moved maximum per row (a vote over
//     the warpgroup; O^T is rescaled only when a score exceeds it by 2^8), P = 2^(z - m + 7) in
//     FP16, the sums of the rounded P in registers until the pair ends.
//   * one warp copies raw tiles (8 groups of 2,304 bytes) into a ring, ahead of everything;
//   * one warp issues the products.
// Tile j + 1 is expanded before the softmax of tile j, whose scores are ready by then, and
// O^T += V^T P^T of tile j runs while tile j + 2 is expanded: K, S, V and P are double.
//
// Split: all pairs' 128-token tiles form one flat range (a pair's start counts as one tile
// more), cut equally over the CTAs of a row tile.  A pair that lies in one CTA is normalised
// and written there; others leave (m, l, O) partials that a second kernel joins.  Tiles wholly
// before the window of every row are left out.  Every wait is bounded.
#include <mutex>

#include "common.cuh"
#include "flat_plan.cuh"
#include "kernels.h"
#include "quantize.cuh"
#include "tcgen05.cuh"

namespace nvfp4kv {

namespace {

constexpr int kWorkersT = 512;                // warps 0 .. 15
constexpr int kThreadsT = kWorkersT + 64;     // + the MMA warp (16) and the load warp (17)
constexpr int kTileT = 128;                   // tokens a tile
constexpr int kBlockT = kTileT * 128;         // bytes of a column block: 64 dims (or rows of P) of 128 tokens
constexpr int kGroupT = 2304;                 // bytes of a 16-token group
constexpr int kRawT = 8 * kGroupT;            // a raw tile
constexpr uint32_t kWaitLimitT = 1u << 24;
constexpr float kNegInfT = -__builtin_huge_valf();
constexpr float kRescaleT = 8.0f;
constexpr float kPOffsetT = 7.0f;             // P = 2^(z - m + 7): at most 2^15
constexpr float kNoMaxT = 3.402823466e38f;    // the offset while every score was -inf
constexpr int kPairUnits = 1;                 // what a pair's start costs a CTA, in tiles

template <int N>
struct TSmem {
    static constexpr int kPBlocks = N == 128 ? 2 : 1;
    static constexpr int kStages = N == 128 ? 3 : 6;
    static constexpr int kQBlock = N * 128;                       // a column block of Q, [N][64]
    static constexpr int kQ = 0;
    static constexpr int kV = 2 * kQBlock > 4096 ? 2 * kQBlock : 4096;
    static constexpr int kP = kV + 2 * 2 * kBlockT;               // V: two tiles of two column blocks
    static constexpr int kRaw = kP + 2 * kPBlocks * kBlockT;      // P: two
    static constexpr int kBar = kRaw + kStages * kRawT;
    // k_full[2] v_full[2] s_done[2] p_full[2] pv_done[2] drain raw_full[] raw_free[]
    static constexpr int kNumBars = 11 + 2 * kStages;
    static constexpr int kMisc = kBar + 8 * kNumBars;             // tmem base, abort, valid[kStages]
    static constexpr int kM = (kMisc + 8 + 4 * kStages + 15) & ~15;   // float m[N], fac[N], alpha[N], off[N], slope[N], depth[N]
    static constexpr int kRow = kM + 6 * N * 4;                   // int row[N] (-1: none), draft[N]
    static constexpr int kWarpMax = kRow + 2 * N * 4;             // float [4][4][N / 4]
    static constexpr int kMask = kWarpMax + 4 * N * 4;            // u64 mask[64], int depth[64]
    static constexpr int kBytes = kMask + 64 * 12;
    // TMEM columns: O at 0, S[2], K[2]
    static constexpr uint32_t kColS = N, kColK = 3 * N, kCols = 512;
    static_assert(kColK + 128 <= kCols, "TMEM columns");
    static_assert(kV % 1024 == 0 && kP % 1024 == 0 && kRaw % 1024 == 0 && kBar % 16 == 0 && kMask % 8 == 0, "alignment");
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static_assert(sizeof(FlatScratch<kThreadsT>) <= 2 * kBlockT, "the plan's scratch lies in the V tile");
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
    float cap_in;             // 2 log2(e) / cap * sm_scale * g_K
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

// The tiles of a CTA's range in order.
struct TreeIter {
    int b, kv, t;    // t: tile of the pair, from 0
    Seq s;
    int left;        // units of the range from this one on
};

__device__ __forceinline__ void next_tile(const TreeArgs &a, TreeIter &it, int r0) {
    it.left--;
    if (++it.t < it.s.nt || it.left <= 0) return;
    it.t = 0;
    it.left -= kPairUnits;
    if (it.left <= 0 || ++it.kv < a.Hkv) return;
    it.kv = 0;
    do {             // left > 0: a later sequence has tiles
        it.s = seq_of(a, ++it.b);
    } while (pair_units(a, it.s, r0) == 0);
}

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const volatile int *abort_flag) {
    for (uint32_t n = 0; n < kWaitLimitT; n++) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 63) == 63 && *abort_flag) return false;
    }
    return false;
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

// OPT: the scores are capped or biased.
template <int N, bool OPT>
__global__ void __launch_bounds__(kThreadsT, 1) tree_kernel(TreeArgs a) {
    using L = TSmem<N>;
    constexpr int CW = N / 4;                     // rows per warpgroup
    constexpr int S = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBar);
    uint64_t *k_full = bars, *v_full = bars + 2, *s_done = bars + 4, *p_full = bars + 6, *pv_done = bars + 8;
    uint64_t *drain = bars + 10, *raw_full = bars + 11, *raw_free = raw_full + S;
    uint32_t &tmem_base = *reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    volatile int *s_valid = abort_flag + 1;
    float *s_m = reinterpret_cast<float *>(smem + L::kM), *s_fac = s_m + N, *s_alpha = s_fac + N, *s_off = s_alpha + N;
    float *s_slope = s_off + N, *s_dep = s_slope + N;
    int *s_row = reinterpret_cast<int *>(smem + L::kRow), *s_draft = s_row + N;
    uint64_t *s_mask = reinterpret_cast<uint64_t *>(smem + L::kMask);
    int *s_depth = reinterpret_cast<int *>(s_mask + 64);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r0 = blockIdx.y * N;
    if (tid == 0) {
        for (int i = 0; i < 4; i++) mbar_init(&bars[i], i < 2 ? kWorkersT / 32 : kWorkersT / 64);
        for (int i = 4; i < 11; i++) mbar_init(&bars[i], i == 6 || i == 7 ? kWorkersT / 32 : 1);
        for (int i = 0; i < S; i++) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_free[i], kWorkersT / 32);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait();               // everything read or written may belong to earlier work of the stream
    pdl_launch_dependents();
    if (warp == 16) tc_alloc(&tmem_base, L::kCols);

    int b0;
    unsigned first, u0 = 0, u1 = 0;
    flat_locate<kThreadsT>(
        *reinterpret_cast<FlatScratch<kThreadsT> *>(smem + L::kV), a.B,
        [&](int b) { return (unsigned)a.Hkv * pair_units(a, seq_of(a, b), r0); },
        [&](unsigned total) {
            const FlatCut cut(total, a.splits);
            u0 = cut.begin(blockIdx.x);
            u1 = cut.begin(blockIdx.x + 1);
            return u0 < u1 ? u0 : kFlatNone;
        },
        b0, first);
    if (warp == 16 && blockIdx.y == 0) {   // what is out of range, and the rows of sequences without tokens
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
    it.left = 0;
    if (u0 < u1) {
        it.s = seq_of(a, b0);
        const int per = it.s.nt + kPairUnits, rel = (int)(u0 - first), in = rel % per;
        it.kv = rel / per;
        it.t = max(0, in - kPairUnits);
        it.left = (int)(u1 - u0) - max(0, kPairUnits - in);
    }
    if (it.left <= 0) {   // a range without tiles
        if (warp == 16) tc_dealloc(tmem_base, L::kCols);
        return;
    }
    const uint32_t tmem = tmem_base, sbase = smem_u32(smem);
    if (warp == 16) {
        // ---------------- the MMA warp: the whole warp runs the loop, one elected lane issues
        constexpr uint32_t idesc_s = idesc_f16_f32(128, N, false);
        constexpr uint32_t idesc_o = idesc_a_mn_major(idesc_f16_f32(128, N, true));
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const bool leader = elect_one();
        // operand descriptors; a step adds its byte offset / 16 to the address field
        const uint64_t dQ = smem_desc_sw128(sbase + L::kQ, 16, 1024);
        const uint64_t dP = smem_desc_sw128(sbase + L::kP, kBlockT, 1024), dV = smem_desc_sw128(sbase + L::kV, kBlockT, 1024);
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            const bool good = __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
            tc_fence_after();
            return good;
        };
        auto scores = [&](uint32_t j) {   // S^T(j), once K(j) (and a pair's Q) has arrived
            const uint32_t buf = j & 1;
            if (!wait(&k_full[buf], (j >> 1) & 1)) return false;
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < 8; kk++)
                    tc_mma_bf16_tmem_a(tm + L::kColS + buf * N, tm + L::kColK + buf * 64 + kk * 8,
                                       dQ + ((kk >> 2) * (L::kQBlock / 16) + (kk & 3) * 2), idesc_s, kk > 0);
                tc_commit(&s_done[buf]);
            }
            return true;
        };
        bool fresh = true, ok = scores(0);
        for (uint32_t j = 0; ok; j++) {
            TreeIter nx = it;
            next_tile(a, nx, r0);
            const bool same = nx.left > 0 && nx.t > 0;      // the next tile belongs to the same pair
            if (same) ok = scores(j + 1);
            const uint32_t buf = j & 1;
            ok = ok && wait(&p_full[buf], (j >> 1) & 1);
            ok = ok && wait(&v_full[buf], (j >> 1) & 1);
            if (!ok) break;
            if (leader) {
                const uint64_t v = dV + buf * (2 * kBlockT / 16), p = dP + buf * (L::kPBlocks * kBlockT / 16);
                const uint32_t acc = fresh ? 0u : 1u;
#pragma unroll
                for (int kk = 0; kk < 8; kk++)   // 16 tokens: 2,048 bytes of a column block, and of P
                    tc_mma_bf16(tm, v + kk * 128, p + kk * 128, idesc_o, kk > 0 ? 1u : acc);
                tc_commit(&pv_done[buf]);
            }
            it = nx;
            fresh = !same;
            if (it.left <= 0) break;
            if (fresh) ok = scores(j + 1);
        }
        if (!ok && leader) {
            if (!*abort_flag) flag_error(a.err, kErrTimeout);
            *abort_flag = 1;
            tc_commit(drain);   // no product may still read the CTA's memory when it ends
            mbar_wait_bounded(drain, 0, kWaitLimitT, nullptr);
        }
        __syncwarp();
    } else if (warp == 17) {
        // ---------------- the load warp: lane g < 8 copies group g of each tile
        uint32_t j = 0;
        int32_t page = -1;
        auto token = [&](const TreeIter &x) { return (x.s.t0 + x.t) * kTileT + 16 * lane; };
        auto page_of = [&](const TreeIter &x) {
            const int t = token(x);
            return x.left > 0 && lane < 8 && t < x.s.n ? __ldg(a.block_table + (int64_t)x.b * a.max_pages + (t >> a.log2P)) : -1;
        };
        page = page_of(it);
        for (; it.left > 0; j++) {
            const uint32_t st = j % S, ph = (j / S) & 1;
            if (j >= S && !__all_sync(0xffffffffu, wait_bar(&raw_free[st], ph ^ 1u, abort_flag))) {
                if (lane == 0 && !*abort_flag) flag_error(a.err, kErrTimeout);
                *abort_flag = 1;
                break;
            }
            const int t = token(it);
            const bool want = lane < 8 && t < it.s.n, good = want && page >= 0 && page < a.num_pages;
            if (want && !good) flag_error(a.err, kErrPage);
            const unsigned mask = __ballot_sync(0xffffffffu, good);
            if (lane == 0) {
                s_valid[st] = (int)mask;
                mbar_arrive_expect_tx(&raw_full[st], (uint32_t)__popc(mask) * kGroupT);
            }
            __syncwarp();
            if (good)
                bulk_g2s(smem + L::kRaw + st * kRawT + lane * kGroupT,
                         a.pool + ((int64_t)page * a.Hkv + it.kv) * a.slab + (int64_t)((t & (a.P - 1)) >> 4) * kGroupT, kGroupT,
                         &raw_full[st]);
            next_tile(a, it, r0);
            page = page_of(it);
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
        const int wg = warp >> 2, row = 32 * (warp & 3) + lane;   // softmax: row quarter, token
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        // expanding: group grp of the tile (its TMEM lanes are this warp's to reach), K or V
        const int grp = 2 * (warp & 3) + (wg & 1), er = lane >> 2, eq = lane & 3;
        const bool is_v = wg >> 1;
        const uint32_t glanes = (uint32_t)(16 * grp) << 16;

        // The raw tile j -> K in TMEM or V in shared memory; returns the groups that it holds.
        auto expand = [&](const TreeIter &x, uint32_t j) {
            const uint32_t st = j % S, buf = j & 1;
            wait(&raw_full[st], (j / S) & 1);
            const int held = s_valid[st];
            const bool landed = (held >> grp) & 1;
            const int rows = landed ? x.s.n - ((x.s.t0 + x.t) * kTileT + 16 * grp) : 0;   // rows of the group that exist
            const uint8_t *g = smem + L::kRaw + st * kRawT + grp * kGroupT;
            if (!is_v) {
                uint32_t f[2][16];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int r = er + 8 * e;
                    const uint4 c = *reinterpret_cast<const uint4 *>(g + r * 64 + eq * 16);
                    const uint32_t s = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(g + 1024 + r * 8 + eq * 2));
                    const uint32_t s0 = __byte_perm(s, 0, 0x1010), s1 = __byte_perm(s, 0, 0x3232);
                    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int m = 0; m < 4; m++) {
                        e2m1x8_to_f16x2x4(w[m], f[e][4 * m], f[e][4 * m + 1], f[e][4 * m + 2], f[e][4 * m + 3]);
#pragma unroll
                        for (int i = 0; i < 4; i++) f[e][4 * m + i] = hmul2(f[e][4 * m + i], m < 2 ? s0 : s1);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&raw_free[st]);
                // (rows that do not exist: their scores are masked, whatever these values are)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    uint32_t v[16];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        v[4 * k] = f[0][8 * h + 2 * k];
                        v[4 * k + 1] = f[0][8 * h + 2 * k + 1];
                        v[4 * k + 2] = f[1][8 * h + 2 * k];
                        v[4 * k + 3] = f[1][8 * h + 2 * k + 1];
                    }
                    tc_st_16x256_x4(tmem + glanes + L::kColK + 64 * buf + 32 * h, v);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&k_full[buf]);
            } else {
                if (lane == 0) mbar_arrive(&k_full[buf]);     // (a pair's Q, stored by all warps)
                uint32_t f[2][16];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int r = er + 8 * e;
                    uint4 c = *reinterpret_cast<const uint4 *>(g + 1152 + r * 64 + eq * 16);
                    uint32_t s = (uint32_t)g[2176 + (2 * eq) * 16 + r] | ((uint32_t)g[2176 + (2 * eq + 1) * 16 + r] << 8);
                    if (r >= rows) {                          // may hold anything: zeros
                        c = make_uint4(0, 0, 0, 0);
                        s = 0;
                    }
                    s = e4m3x2_to_f16x2(s);
                    uint32_t s0 = __byte_perm(s, 0, 0x1010), s1 = __byte_perm(s, 0, 0x3232);
                    // lanes q >= 2 store their words 2, 3, 0, 1, so that a quarter warp meets all banks
                    const bool sw = eq & 2;
                    const uint32_t w[4] = {sw ? c.z : c.x, sw ? c.w : c.y, sw ? c.x : c.z, sw ? c.y : c.w};
                    if (sw) {
                        const uint32_t x0 = s0;
                        s0 = s1;
                        s1 = x0;
                    }
#pragma unroll
                    for (int m = 0; m < 4; m++) {
                        e2m1x8_to_f16x2x4(w[m], f[e][4 * m], f[e][4 * m + 1], f[e][4 * m + 2], f[e][4 * m + 3]);
#pragma unroll
                        for (int i = 0; i < 4; i++) f[e][4 * m + i] = hmul2(f[e][4 * m + i], m < 2 ? s0 : s1);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&raw_free[st]);
                if (j >= 2) wait(&pv_done[buf], ((j >> 1) - 1) & 1);
                uint8_t *blk = smem + L::kV + (2 * buf + (eq >> 1)) * kBlockT;
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int tr = 16 * grp + er + 8 * e;
#pragma unroll
                    for (int m = 0; m < 4; m++)
                        *reinterpret_cast<uint4 *>(blk + sw128_off(tr, (eq & 1) * 4 + (m ^ (eq & 2)))) =
                            make_uint4(f[e][4 * m], f[e][4 * m + 1], f[e][4 * m + 2], f[e][4 * m + 3]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_full[buf]);
            }
            return held;
        };
        // A pair's Q, the rows' factors and the tree.  (The previous pair's products and its
        // epilogue are done.)
        auto load_pair = [&](const TreeIter &x) {
            const int rows = x.s.d * a.G;
#pragma unroll 2
            for (int k = 0; k < N / 16; k++) {
                const int c = warp + 16 * k, r = r0 + c;
                const int i = r / a.G, h = x.kv * a.G + (r - i * a.G);
                uint2 w = make_uint2(0, 0);
                if (r < rows) w = __ldg(reinterpret_cast<const uint2 *>(a.q + ((int64_t)(x.s.q0 + i) * a.Hq + h) * kHeadDim) + lane);
                uint32_t m = max_u16x2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
                m = __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xffffu));
                // 2^kq puts the row's largest value into [2^14, 2^15)
                const int kq = m ? min(126, max(-126, 14 - ((int)(m >> 7) - 127))) : 0;
                const float sc = __uint_as_float((uint32_t)(kq + 127) << 23);
                // dims 4 lane .. + 3 = 32 q + 4 a + e lie at position 16 a + 4 q + e
                const int pos = 16 * (lane & 7) + 4 * (lane >> 3);
                *reinterpret_cast<uint2 *>(smem + L::kQ + (pos >> 6) * L::kQBlock + sw128_off(c, (pos & 63) >> 3) + (pos & 7) * 2) =
                    make_uint2(f32x2_to_f16x2(bf16_hi(w.x) * sc, bf16_lo(w.x) * sc),
                               f32x2_to_f16x2(bf16_hi(w.y) * sc, bf16_lo(w.y) * sc));
                if (lane == 0) {
                    s_fac[c] = (OPT && a.cap_log2 > 0.f ? a.cap_in : a.score_log2) * __uint_as_float((uint32_t)(127 - kq) << 23);
                    s_m[c] = kNegInfT;
                    s_off[c] = kNoMaxT;
                    s_row[c] = r < rows ? (x.s.q0 + i) * a.Hq + h : -1;
                    s_draft[c] = min(i, 63);
                    if (OPT) s_slope[c] = a.slopes && r < rows ? __ldg(a.slopes + h) * 1.4426950408889634f : 0.f;
                }
            }
            if (tid < 64) {
                const uint64_t all = x.s.d >= 64 ? ~0ull : (1ull << x.s.d) - 1;
                uint64_t mk = 0;
                if (tid < x.s.d) mk = (a.mask ? a.mask[x.s.q0 + tid] : (2ull << tid) - 1) & all;
                s_mask[tid] = mk;
                s_depth[tid] = __popcll(mk) - 1;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // Q for the tensor core
            workers_sync();
            if (OPT) {
                if (tid < N) s_dep[tid] = (float)s_depth[s_draft[tid]];
                workers_sync();
            }
        };

        bool fresh = true;                      // the range's first tile of its pair
        int t_begin = it.t;
        float l[CW];
        load_pair(it);
        int held = 0, held_next = expand(it, 0);
        for (uint32_t j = 0; it.left > 0; j++) {
            const uint32_t buf = j & 1;
            if (fresh) {
                if (j > 0) {
                    load_pair(it);
                    held_next = expand(it, j);
                }
#pragma unroll
                for (int c = 0; c < CW; c++) l[c] = 0.f;
            }
            TreeIter nx = it;
            next_tile(a, nx, r0);
            const bool same = nx.left > 0 && nx.t > 0;
            // (K's buffer of tile j + 1 is free: the scores of tile j - 1 were seen)
            held = held_next;
            if (same) held_next = expand(nx, j + 1);

            // ---- softmax of the token's scores for the warpgroup's rows
            const int tok0 = (it.s.t0 + it.t) * kTileT, tok = tok0 + row;
            // edge: a token of the tile that some row does not see
            const bool edge = tok0 + kTileT > it.s.base || (a.window > 0 && tok0 <= it.s.n - 1 - a.window) ||
                              held != 0xff;
            uint32_t gone = 0;                  // bit c: row c of the warpgroup does not see the token
            const int rel = tok - it.s.base;
            int key = rel;                      // the token's position, from base on
            if (edge || OPT) {
                const int jj = rel < 0 ? 0 : min(rel, 63);
                if (rel >= 0) key = s_depth[jj];
                if (edge) {
                    const bool there = tok < it.s.n && ((held >> (row >> 4)) & 1);
#pragma unroll 4
                    for (int c = 0; c < CW; c++) {
                        const int i = s_draft[wg * CW + c];
                        const bool sees = there && (rel < 0 || (s_mask[i] >> jj) & 1) &&
                                          (a.window <= 0 || key > s_depth[i] - a.window);
                        gone |= sees ? 0u : 1u << c;
                    }
                }
            }
            wait(&s_done[buf], (j >> 1) & 1);
            tc_fence_after();
            // d = z - m + 7 in base 2
            float d[CW];
            auto score = [&](uint32_t s, int c) {    // z (OPT), without the row's offset
                float z = __uint_as_float(s) * s_fac[wg * CW + c];
                if (OPT) {
                    if (a.cap_log2 > 0.f) {          // cap tanh(x) = cap - 2 cap / (1 + e^(2 x))
                        const float e = ex2(z) + 1.0f;
                        z = fmaf(-2.0f * a.cap_log2, rcp_approx(e), a.cap_log2);
                    }
                    z = fmaf(s_slope[wg * CW + c], (float)key - s_dep[wg * CW + c], z);
                }
                return z;
            };
            auto load_scores = [&]() {
                uint32_t sr[CW];
                load_columns<CW>(tmem + lanes + L::kColS + buf * N + wg * CW, sr);
                tc_wait_ld();
                const float4 *fac = reinterpret_cast<const float4 *>(s_fac + wg * CW);
                const float4 *off = reinterpret_cast<const float4 *>(s_off + wg * CW);
#pragma unroll
                for (int x = 0; x < CW / 4; x++) {
                    const float4 o = off[x];
                    if (OPT) {
                        d[4 * x] = score(sr[4 * x], 4 * x) + o.x;
                        d[4 * x + 1] = score(sr[4 * x + 1], 4 * x + 1) + o.y;
                        d[4 * x + 2] = score(sr[4 * x + 2], 4 * x + 2) + o.z;
                        d[4 * x + 3] = score(sr[4 * x + 3], 4 * x + 3) + o.w;
                    } else {
                        const float4 f = fac[x];
                        d[4 * x] = fmaf(__uint_as_float(sr[4 * x]), f.x, o.x);
                        d[4 * x + 1] = fmaf(__uint_as_float(sr[4 * x + 1]), f.y, o.y);
                        d[4 * x + 2] = fmaf(__uint_as_float(sr[4 * x + 2]), f.z, o.z);
                        d[4 * x + 3] = fmaf(__uint_as_float(sr[4 * x + 3]), f.w, o.w);
                    }
                }
                if (edge) {
#pragma unroll
                    for (int c = 0; c < CW; c++)
                        if ((gone >> c) & 1) d[c] = kNegInfT;
                }
            };
            load_scores();
            float top = d[0];
#pragma unroll
            for (int c = 1; c < CW; c++) top = fmaxf(top, d[c]);
            if (group_any(wg, top > kRescaleT + kPOffsetT)) {
                float *wmax = reinterpret_cast<float *>(smem + L::kWarpMax) + wg * 4 * CW;
                int mine = 0;
                uint32_t sr[CW];
                load_columns<CW>(tmem + lanes + L::kColS + buf * N + wg * CW, sr);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < CW; c++) {
                    const float z = (gone >> c) & 1 ? kNegInfT : score(sr[c], c);
                    const int mx = __reduce_max_sync(0xffffffffu, ordered(z));
                    if (lane == c) mine = mx;
                }
                if (lane < CW) wmax[(warp & 3) * CW + lane] = unordered(mine);
                group_sync(wg);
                if ((warp & 3) == 0 && lane < CW) {
                    const float mx = fmaxf(fmaxf(wmax[lane], wmax[CW + lane]), fmaxf(wmax[2 * CW + lane], wmax[3 * CW + lane]));
                    const float mo = s_m[wg * CW + lane], mn = fmaxf(mo, mx);
                    s_alpha[wg * CW + lane] = mo == kNegInfT ? 0.f : ex2(mo - mn);
                    s_m[wg * CW + lane] = mn;
                    s_off[wg * CW + lane] = mn == kNegInfT ? kNoMaxT : kPOffsetT - mn;
                }
                group_sync(wg);
#pragma unroll
                for (int c = 0; c < CW; c++) l[c] *= s_alpha[wg * CW + c];
                if (!fresh) {   // O^T holds the earlier tiles: rescale the warpgroup's rows
                    wait(&pv_done[buf ^ 1], ((j - 1) >> 1) & 1);
                    tc_fence_after();
                    uint32_t ov[CW];
                    load_columns<CW>(tmem + lanes + wg * CW, ov);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < CW; c++) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * s_alpha[wg * CW + c]);
                    if constexpr (CW == 32) tc_st32(tmem + lanes + wg * CW, ov);
                    else tc_st(tmem + lanes + wg * CW, ov);
                    tc_wait_st();
                }
                load_scores();
            }
            if (j >= 2) wait(&pv_done[buf], ((j >> 1) - 1) & 1);     // P's buffer is free
            uint8_t *pt = smem + L::kP + (buf * L::kPBlocks + (wg * CW) / 64) * kBlockT;
#pragma unroll
            for (int c0 = 0; c0 < CW; c0 += CW < 8 ? CW : 8) {
                uint32_t pw[4];
#pragma unroll
                for (int e = 0; e < (CW < 8 ? CW : 8) / 2; e++) {
                    pw[e] = f32x2_to_f16x2(ex2(d[c0 + 2 * e + 1]), ex2(d[c0 + 2 * e]));
                    add_f16x2(l[c0 + 2 * e], l[c0 + 2 * e + 1], pw[e]);
                }
                if (CW == 4)   // eight bytes a thread: two warpgroups share a 16-byte chunk
                    *reinterpret_cast<uint2 *>(pt + sw128_off(row, wg >> 1) + (wg & 1) * 8) = make_uint2(pw[0], pw[1]);
                else
                    *reinterpret_cast<uint4 *>(pt + sw128_off(row, ((wg * CW + c0) & 63) / 8)) =
                        make_uint4(pw[0], pw[1], pw[2], pw[3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[buf]);

            // ---- the pair's last tile of this range: normalise, or leave the partial
            const TreeIter cur = it;
            it = nx;
            fresh = !same;
            if (!fresh) continue;
            wait(&pv_done[buf], (j >> 1) & 1);
            tc_fence_after();
            {
                float *wsum = reinterpret_cast<float *>(smem + L::kWarpMax) + wg * 4 * CW;
                const float s = column_sums<CW>(l, lane);
                if (lane < CW) wsum[(warp & 3) * CW + lane] = s;
                group_sync(wg);
                const bool whole = t_begin == 0 && cur.t == cur.s.nt - 1;
                const int64_t slot = (int64_t)blockIdx.y * ((int64_t)a.splits + (int64_t)a.B * a.Hkv) + blockIdx.x +
                                     (int64_t)cur.b * a.Hkv + cur.kv;
                auto sum = [&](int c) { return (wsum[c] + wsum[CW + c]) + (wsum[2 * CW + c] + wsum[3 * CW + c]); };
                if (!whole && (warp & 3) == 0 && lane < CW) {
                    const float m = s_m[wg * CW + lane];
                    a.part_ml[slot * N + wg * CW + lane] = make_float2(m == kNegInfT ? m : m - kPOffsetT, sum(lane));
                }
                uint32_t ov[CW];
                load_columns<CW>(tmem + lanes + wg * CW, ov);
                tc_wait_ld();
                if (whole) {
#pragma unroll
                    for (int c = 0; c < CW; c++) {
                        const int at = s_row[wg * CW + c];
                        const float t = sum(c), inv = t == 0.f ? 0.f : a.gv / t;   // (a row that sees nothing: zeros)
                        if (at >= 0) a.out[(int64_t)at * kHeadDim + row] = __float2bfloat16_rn(__uint_as_float(ov[c]) * inv);
                    }
                } else {
                    float *dst = a.part_acc + (slot * N + wg * CW) * kHeadDim + row;
#pragma unroll
                    for (int c = 0; c < CW; c++)
                        if (s_row[wg * CW + c] >= 0) dst[c * kHeadDim] = __uint_as_float(ov[c]);
                }
                tc_fence_before();
                workers_sync();   // sums, maxima and rows are read: the next pair may write them
            }
            t_begin = it.t;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) tc_dealloc(tmem, L::kCols);
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
            // (a partial without a maximum counts nothing, unless its sum is NaN)
            const float f = ml[k].x == kNegInfT ? (ml[k].y == 0.f ? 0.f : ml[k].y) : ex2(ml[k].x - mx);
            if (f == 0.f) continue;
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
    int smem;
};

template <int N>
TreeFns fns_of() {
    return {{reinterpret_cast<const void *>(&tree_kernel<N, false>), reinterpret_cast<const void *>(&tree_kernel<N, true>)},
            reinterpret_cast<const void *>(&tree_join_kernel<N>), TSmem<N>::kBytes};
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
    return sms / tiles > 0 ? (int)(sms / tiles) : 1;
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
    a.cap_log2 = (float)(softcap * log2e);
    a.cap_in = softcap > 0.f ? (float)(2.0 * log2e * scale / softcap) : 0.f;
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
    const bool opt = softcap > 0.f || slopes;
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
    e = launch_pdl(f.tree[opt], dim3((unsigned)a.splits, (unsigned)tiles), kThreadsT, (size_t)f.smem, stream, args);
    if (e != cudaSuccess || a.splits == 1 || a.cap <= kTileT) return e;   // no pair can have been split
    return launch_pdl(f.join, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps), (unsigned)a.Hkv, (unsigned)batch),
                      32 * kJoinWarps, 0, stream, args);
}

}  // namespace nvfp4kv
