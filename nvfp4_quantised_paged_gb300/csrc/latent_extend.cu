// latent_extend.cu -- expanded latent attention of a chunk over [expanded prefix || expanded chunk].
//
//   out[t][h] = sum_j softmax_j(sm_scale (q[t][h][:128] . k_j[h] + q[t][h][128:] . r_j)) v_j[h],
// causal in the chunk: the form a prefill takes, where the latents' up-projection
// to per-head K and V (a library GEMM on the rows that the dequant kernel writes)
// is shared by many queries.  The 64 rotary key values r_j are one row for all
// heads and are never copied per head.
//
// The pipeline is extend_attention.cu's: one CTA = 256 chunk tokens of one head in
// two 128-row query tiles, one softmax warpgroup each with one row (= TMEM lane) a
// thread; a warp per query tile issues its tcgen05 products, two independent chains that
// the tensor core overlaps.  What differs:
//   * S_w = Q_w K^T takes twelve K 16 steps, eight over K's two column blocks and
//     four over the rotary block, a third one that its own tensor map fills; a
//     query tile is 48 KB, and a K/V tile 80 KB in five column blocks;
//   * Q leaves room for eight blocks of 16 KB, not for two K/V tiles: they are a
//     ring that the load warp fills in the order K(j) K(j) R(j) V(j) V(j) K(j + 1) ...,
//     each slot as soon as the products that read it are done (whole slots of one
//     V and two K tiles left V's load on the critical path: 277 us against
//     212 us for 4 x 512 tokens over up to 8,192, 32 heads).  V's two blocks
//     need not be neighbours: O_w += P_w V runs as two N 64 products a step, which
//     with P in TMEM cost what one of N 128 does (30 and 60 clocks);
//   * rows of a V tile past the request's end are zeroed in shared memory before
//     the product: they are other requests' rows or padding, and a NaN there times
//     a probability of 0 would still be a NaN.
// Bound by the tensor cores: 2 * (192 + 128) flops a (query, key, head), K and V
// tiles shared by 256 queries through L2.  Every wait is bounded.
#include <cooperative_groups.h>

#include <mutex>

#include "common.cuh"
#include "extend_common.cuh"
#include "kernels.h"
#include "latent.cuh"
#include "tcgen05.cuh"

namespace nvfp4kv {

namespace {

namespace cg = cooperative_groups;

constexpr int kWGs = 2;
constexpr int kQRows = 128;
constexpr int kCtaRows = kWGs * kQRows;
constexpr int kSoftThreads = kWGs * kQRows;
constexpr int kEThreads = kSoftThreads + 64;   // + the MMA warp and the load warp
constexpr int kKeys = 128;
constexpr int kQkDim = kHeadDim + kRopeDim;    // 192
constexpr int kBlockBytes = 128 * 128;         // one column block: 128 rows of 64 BF16 values
constexpr int kQBytes = 3 * kBlockBytes;
constexpr int kSlots = 8;                      // ring of column blocks: block 5 t + i of tile t (i = 0 1: K, 2: rotary, 3 4: V)
constexpr int kOffQ = 0;
constexpr int kOffRing = kWGs * kQBytes;
constexpr int kOffBar = kOffRing + kSlots * kBlockBytes;
constexpr int kNumBars = kSlots + 11;          // k_full[2] v_full[2] empty[8] s_done[2] p_full[2] pv_done[2] drain
constexpr int kOffTmem = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kOffOrder = kOffBar + 256;       // int[256]: requests by decreasing prefix length
constexpr int kOrderMax = 256;
constexpr int kMaxSplit = 8;                   // CTAs of a cluster
constexpr int kESmem = kOffOrder + 4 * kOrderMax;
static_assert(kOffAbort + 4 <= kOffOrder && kESmem <= 227 * 1024, "shared memory of a CTA");
// TMEM columns: S_w at 128w (FP32; P_w as BF16 pairs over its first 64 columns), O_w at 256 + 128w
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr float kRescale = 8.0f;
constexpr float kNegInfE = -__builtin_huge_valf();

struct ExtendArgs {
    const uint16_t *q;                 // BF16 [total_q][H][192]
    const int32_t *cu_prefix, *cu_q;
    int H, max_q_len;
    int64_t total_q, total_prefix;
    float score_log2;                  // sm_scale * log2(e), positive
    uint16_t *out;                     // BF16 [total_q][H][128]
    unsigned *err;
};

constexpr int kMinTiles = 4;                   // K/V tiles from which on clusters share them

// K/V as 3-D maps [rows][heads][128] (any strides), the rotary rows as [rows][1][64]; boxes of 64 x 1 x 128.
struct ExtendMaps {
    CUtensorMap k_pre, v_pre, r_pre, k_new, v_new, r_new;
};

// Bounded wait that polls without suspending the thread (these waits are on the critical path).
__device__ __forceinline__ bool poll_wait(uint64_t *bar, uint32_t parity, const volatile int *abort_flag) {
    for (uint32_t n = 0; n < 4 * kWaitLimitE; n++) {
        if (mbar_test_wait(bar, parity)) return true;
        if ((n & 255) == 255 && *abort_flag) return false;
    }
    return false;
}

__global__ void __launch_bounds__(kEThreads, 1)
    latent_extend_kernel(const __grid_constant__ ExtendMaps maps, ExtendArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *k_full = bars, *v_full = bars + 2, *empty = bars + 4, *s_done = empty + kSlots, *p_full = s_done + 2;
    uint64_t *pv_done = p_full + 2, *drain = pv_done + 2;
    uint32_t &tmem_base = *reinterpret_cast<uint32_t *>(smem + kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffAbort);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();               // everything read or written may belong to earlier work of the stream
    pdl_launch_dependents();
    // Requests in order of decreasing prefix length: blockIdx.z is the rank (the longest CTAs start first).
    int r = blockIdx.z;
    if (gridDim.z <= kOrderMax) {
        int *order = reinterpret_cast<int *>(smem + kOffOrder);
        const int nr = (int)gridDim.z;
        auto prefix_len = [&](int c) { return a.cu_prefix[c + 1] - a.cu_prefix[c]; };
        if (tid < nr) {
            const int nj = prefix_len(tid);
            int rank = 0;
            for (int c = 0; c < nr; c++) {
                const int nc = prefix_len(c);
                rank += nc > nj || (nc == nj && c < tid);
            }
            order[rank] = tid;
        }
        __syncthreads();
        r = order[blockIdx.z];
    }
    const int head = blockIdx.y;
    const int q0 = a.cu_q[r], p0 = a.cu_prefix[r];
    int L = a.cu_q[r + 1] - q0;
    const int np = a.cu_prefix[r + 1] - p0;
    const bool first_cta = tid == 0 && blockIdx.x == 0 && head == 0;
    // a request outside the rows that the caller says there are is skipped
    if (L < 0 || np < 0 || q0 < 0 || p0 < 0 || (int64_t)q0 + L > a.total_q || (int64_t)p0 + np > a.total_prefix) {
        if (first_cta) flag_error(a.err, kErrCuPrefix);
        return;
    }
    if (L > a.max_q_len) {
        if (first_cta) flag_error(a.err, kErrSeqLen);
        L = a.max_q_len;
    }
    // A cluster of C CTAs shares the query rows; each takes a contiguous part of the K/V tiles.
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row0 = (int)(blockIdx.x / C) * kCtaRows;
    if (row0 >= L) return;                                      // (all of the cluster)
    const int nwg = row0 + kQRows < L ? 2 : 1;                  // query tiles holding rows
    const int t_last = min(row0 + kCtaRows, L) - 1;             // last chunk token of this CTA
    const int nt_pre = (np + kKeys - 1) / kKeys;
    const int nt_all = nt_pre + t_last / kKeys + 1;
    const int j0 = (int)((int64_t)nt_all * rank / C), nt = (int)((int64_t)nt_all * (rank + 1) / C) - j0;
    const uint32_t sbase = smem_u32(smem);

    // ---- query tiles: 128 rows x 24 chunks of 16 bytes each, by their warpgroups
    if (tid < kSoftThreads) {
        const int w = tid >> 7, t = tid & 127;
        const uint32_t sQ = sbase + kOffQ + w * kQBytes;
#pragma unroll 4
        for (int it = 0; it < 24; it++) {
            const int idx = t + it * kQRows;
            const int row = idx / 24, c16 = idx % 24;
            const int R = row0 + w * kQRows + row;
            const bool ok = R < L;
            const int64_t src = ok ? (((int64_t)q0 + R) * a.H + head) * kQkDim + c16 * 8 : 0;
            cp_async16(sQ + (c16 >> 3) * kBlockBytes + sw128_off(row, c16 & 7), a.q + src, ok);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    auto tile_row = [&](int j) { return j < nt_pre ? p0 + j * kKeys : q0 + (j - nt_pre) * kKeys; };
    auto slot_of = [](uint32_t blk) { return blk % kSlots; };   // (fewer than 2^27 blocks: lengths are int32)
    auto phase_of = [](uint32_t blk) { return (blk / kSlots) & 1u; };

    if (warp == 0) tc_alloc(&tmem_base, kTmemCols);
    if (tid == kSoftThreads) {
        for (int j = 0; j < kNumBars; j++)
            mbar_init(&bars[j], &bars[j] >= empty && &bars[j] < s_done ? nwg : &bars[j] >= p_full && &bars[j] < pv_done ? kQRows : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // Q for the tensor core
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;

    if (warp == kSoftThreads / 32) {
        // ---------------- MMA warp: the whole warp runs the loop and one elected lane
        // issues, so that descriptors stay uniform values (issued under a divergent branch a
        // product cost more than the tensor core's 64 clocks for it)
        {
            constexpr uint32_t idesc_s = idesc_bf16_f32(128, kKeys, false);
            constexpr uint32_t idesc_o = idesc_bf16_f32(128, 64, true);
            auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
            const uint32_t tm = uniform(tmem);
            const bool leader = elect_one();
            const uint64_t dQ = smem_desc_sw128(sbase + kOffQ, 16, 1024);
            const uint64_t dB = smem_desc_sw128(sbase + kOffRing, 16, 1024);   // slot 0, K-major and MN-major alike
            auto mma_s = [&](int w, uint32_t blk) {  // S_w = Q_w K^T over 192 dimensions, 16 at a time
                if (!leader) return;
#pragma unroll
                for (int i = 0; i < 3; i++) {
                    const uint32_t slot = slot_of(blk + i);
                    const uint64_t q = dQ + (w * (kQBytes / 16) + i * (kBlockBytes / 16)), k = dB + slot * (kBlockBytes / 16);
#pragma unroll
                    for (int kk = 0; kk < 4; kk++)
                        tc_mma_bf16(tm + 128u * w, q + kk * 2, k + kk * 2, idesc_s, i + kk > 0);
                    tc_commit(&empty[slot]);
                }
                tc_commit(&s_done[w]);
            };
            auto mma_pv = [&](int w, uint32_t blk, uint32_t acc) {  // O_w += P_w V over 128 keys, 64 dimensions at a time
                if (!leader) return;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const uint32_t slot = slot_of(blk + 3 + i);
                    const uint64_t v = dB + slot * (kBlockBytes / 16);
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)  // P from TMEM: 8 columns = 16 keys
                        tc_mma_bf16_tmem_a(tm + kColO + 128u * w + 64u * i, tm + 128u * w + kk * 8, v + kk * 128, idesc_o,
                                           kk > 0 ? 1u : acc);
                    tc_commit(&empty[slot]);
                }
                tc_commit(&pv_done[w]);
            };
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                const bool good = __all_sync(0xffffffffu, poll_wait(bar, parity, abort_flag));
                tc_fence_after();
                return good;
            };
            // The two query tiles take turns: O_0 += P_0(t) V(t), S_0(t + 1), O_1 += P_1(t) V(t),
            // S_1(t + 1), so the softmax of one runs while the tensor core works for the other
            // (issued as they became ready, the two fell into step and left it idle meanwhile).
            // S_w(t + 1) goes over the columns of P_w(t) and waits for the product that reads
            // it; whether the next K and V have landed is checked while that product runs.
            bool ok = nt == 0 || wait(&k_full[0], 0);
            if (ok && nt > 0) {
                mma_s(0, 0);
                if (nwg > 1) mma_s(1, 0);
            }
            ok = ok && (nt == 0 || wait(&v_full[0], 0));
            for (uint32_t t = 0, blk = 0; ok && t < (uint32_t)nt; t++, blk += 5) {
                const bool more = t + 1 < (uint32_t)nt;
#pragma unroll
                for (int w = 0; w < kWGs; w++) {
                    if (w >= nwg) break;
                    ok = ok && wait(&p_full[w], t & 1);
                    if (ok) mma_pv(w, blk, t > 0 ? 1u : 0u);
                    if (!more) continue;
                    if (w == 0) ok = ok && wait(&k_full[(t + 1) & 1], ((t + 1) >> 1) & 1);
                    if (w == nwg - 1) ok = ok && wait(&v_full[(t + 1) & 1], ((t + 1) >> 1) & 1);
                    ok = ok && wait(&pv_done[w], t & 1);
                    if (ok) mma_s(w, blk + 5);
                }
            }
            if (!ok && leader) {
                if (!*abort_flag) flag_error(a.err, kErrTimeout);
                *abort_flag = 1;
                tc_commit(drain);   // no product may still be running when the CTA frees its memory
                mbar_wait_bounded(drain, 0, kWaitLimitE, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == kSoftThreads / 32 + 1) {
        // ---------------- load warp: the blocks in order, each slot once its readers are done
        const bool leader = elect_one();
        uint32_t blk = 0;
        bool ok = true;
        for (int j = 0; ok && j < nt; j++) {
            const bool pre = j0 + j < nt_pre;
            const CUtensorMap *mk = pre ? &maps.k_pre : &maps.k_new, *mr = pre ? &maps.r_pre : &maps.r_new;
            const CUtensorMap *mv = pre ? &maps.v_pre : &maps.v_new;
            for (int i = 0; i < 5; i++, blk++) {
                const uint32_t slot = slot_of(blk);
                if (blk >= kSlots) {
                    ok = __all_sync(0xffffffffu, spin_wait(&empty[slot], phase_of(blk - kSlots), abort_flag));
                    if (!ok) break;
                }
                uint64_t *full = i < 3 ? &k_full[j & 1] : &v_full[j & 1];   // K and rotary blocks complete one phase, V's the other
                if (leader) {
                    if (i == 0 || i == 3) mbar_arrive_expect_tx(full, (i == 0 ? 3 : 2) * kBlockBytes);
                    tma_load_3d(sbase + kOffRing + slot * kBlockBytes, i < 2 ? mk : i == 2 ? mr : mv,
                                i == 1 || i == 4 ? 64 : 0, i == 2 ? 0 : head, tile_row(j0 + j), full);
                }
                __syncwarp();
            }
        }
        if (!ok && leader) {
            if (!*abort_flag) flag_error(a.err, kErrTimeout);
            *abort_flag = 1;
        }
        // After an abort: request what is missing of the last K or V (its barrier counts whole
        // ones; the slots' contents no longer matter).
        if (!ok) {
            const uint32_t j = blk / 5;
            const bool pre = j0 + (int)j < nt_pre;
            for (uint32_t i = blk % 5; i != 0 && i != 3 && i < 5; i++) {
                uint64_t *full = i < 3 ? &k_full[j & 1] : &v_full[j & 1];
                const CUtensorMap *m = i < 2 ? (pre ? &maps.k_pre : &maps.k_new) : i == 2 ? (pre ? &maps.r_pre : &maps.r_new)
                                                                                       : (pre ? &maps.v_pre : &maps.v_new);
                if (leader)
                    tma_load_3d(sbase + kOffRing + slot_of(5u * j + i) * kBlockBytes, m, i == 1 || i == 4 ? 64 : 0,
                                i == 2 ? 0 : head, tile_row(j0 + (int)j), full);
                blk++;
            }
        }
        // Whichever warp gave up, every copy has landed before the CTA's memory is freed.
        for (uint32_t x = blk > 10 ? blk - 10 : 0; x < blk; x++) {
            const uint32_t t = x / 5;
            if (x % 5 == 0) mbar_wait_bounded(&k_full[t & 1], (t >> 1) & 1, kWaitLimitE, nullptr);
            if (x % 5 == 3) mbar_wait_bounded(&v_full[t & 1], (t >> 1) & 1, kWaitLimitE, nullptr);
        }
    } else if ((tid >> 7) < nwg) {
        // ---------------- softmax of this thread's query row
        const int w = tid >> 7;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;  // this warp's TMEM lanes
        const uint32_t colS = 128u * w, colO = kColO + 128u * w;
        const int token = row0 + w * kQRows + (tid & 127);
        const bool row_ok = token < L;
        float m_run = kNegInfE, l_run = 0.f;
        bool ok = true;
        for (int j = 0; j < nt; j++) {
            // S_w(j) done; its commit also covers O_w += P_w(j - 1) V(j - 1)
            ok = __all_sync(0xffffffffu, poll_wait(&s_done[w], (uint32_t)(j & 1), abort_flag));
            if (!ok) break;
            tc_fence_after();
            const bool pre = j0 + j < nt_pre;
            const int base = pre ? (j0 + j) * kKeys : (j0 + j - nt_pre) * kKeys;
            const int visible = (pre ? np : token + 1) - base;   // keys [0, visible) of the tile are seen
            const bool edge = __any_sync(0xffffffffu, visible < kKeys);  // mask on edge tiles only
            // the row's 64 scores of half h (masked scores are -inf)
            auto load_half = [&](int h, float (&sc)[64]) {
                uint32_t sr[2][32];
                tc_ld32(tmem + lane_base + colS + 64 * h, sr[0]);
                tc_ld32(tmem + lane_base + colS + 64 * h + 32, sr[1]);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 64; c++) sc[c] = __uint_as_float(sr[c >> 5][c & 31]);
                if (edge) {
#pragma unroll
                    for (int c = 0; c < 64; c++)
                        if (64 * h + c >= visible) sc[c] = kNegInfE;
                }
            };
            // P = 2^(s * scale - m) of one half, rounded to BF16 pairs; ls += the rounded values
            auto make_p = [&](const float (&sc)[64], float neg_m, uint32_t (&pw)[32], float (&ls)[4]) {
#pragma unroll
                for (int c = 0; c < 32; c++) {
                    const float2 e = fma2(make_float2(sc[2 * c], sc[2 * c + 1]), a.score_log2, neg_m);
                    const __nv_bfloat162 pr = __floats2bfloat162_rn(ex2(e.x), ex2(e.y));
                    pw[c] = *reinterpret_cast<const uint32_t *>(&pr);
                    add_bf16x2(ls[2 * (c & 1)], ls[2 * (c & 1) + 1], pw[c]);
                }
            };
            auto half_max = [&](const float (&sc)[64]) {
                float m8[8];
#pragma unroll
                for (int e = 0; e < 8; e++) m8[e] = max3(sc[e], sc[8 + e], sc[16 + e]);
#pragma unroll
                for (int e = 0; e < 8; e++) m8[e] = max3(m8[e], sc[24 + e], sc[32 + e]);
#pragma unroll
                for (int e = 0; e < 8; e++) m8[e] = max3(m8[e], sc[40 + e], sc[48 + e]);
#pragma unroll
                for (int e = 0; e < 8; e++) m8[e] = fmaxf(m8[e], sc[56 + e]);
                return max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
            };
            // One pass with the running max as it stands (the lazy rescale lets it
            // lag the true max by up to 2^8): P of half 0 stays in registers until
            // half 1 shows whether the max must move; only then does it go over the
            // scores in TMEM.  If it must (the first tile, rarely later), O and the
            // row sum are rescaled and P is formed again from the scores in TMEM.
            // (a row that has seen no key yet, its part of the tiles lying behind it, has the
            // maximum -inf: its probabilities are 2^(-inf - 0) = 0)
            auto neg_m = [&]() { return m_run == kNegInfE ? 0.f : -m_run; };
            uint32_t pw0[32], pw1[32];
            float ls[4] = {0.f, 0.f, 0.f, 0.f};
            float smax;
            {
                float sc[64];
                load_half(0, sc);
                smax = half_max(sc);
                make_p(sc, neg_m(), pw0, ls);
                load_half(1, sc);
                smax = fmaxf(smax, half_max(sc));
                const float mx = smax * a.score_log2;  // the scale is positive
                const bool need = mx > m_run + kRescale;
                if (!__any_sync(0xffffffffu, need)) {
                    make_p(sc, neg_m(), pw1, ls);
                } else {
                    const float m_new = need ? fmaxf(m_run, mx) : m_run;
                    const float alpha = need ? (m_run == kNegInfE ? 0.f : ex2(m_run - m_new)) : 1.f;
                    if (j > 0) {  // O_w holds tiles 0 .. j - 1 (complete): rescale this warp's rows
#pragma unroll
                        for (int cblk = 0; cblk < 4; cblk++) {
                            uint32_t ov[32];
                            tc_ld32(tmem + lane_base + colO + 32 * cblk, ov);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; e++) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                            tc_st32(tmem + lane_base + colO + 32 * cblk, ov);
                        }
                        tc_wait_st();
                    }
                    l_run *= alpha;
                    m_run = m_new;
                    ls[0] = ls[1] = ls[2] = ls[3] = 0.f;
                    make_p(sc, neg_m(), pw1, ls);
                    load_half(0, sc);
                    make_p(sc, neg_m(), pw0, ls);
                }
            }
            l_run += (ls[0] + ls[1]) + (ls[2] + ls[3]);
            tc_st32(tmem + lane_base + colS, pw0);       // over scores 0 .. 31 (read already)
            tc_st32(tmem + lane_base + colS + 32, pw1);  // over scores 32 .. 63
            tc_wait_st();
            // Rows of V past the request's end (edge tiles only) become zeros once V(j) has
            // landed.  Both warpgroups write them, each before its own product.
            const int there = (pre ? np : L) - base;   // rows of the tile that belong to the request
            if (there < kKeys) {
                const uint32_t blk = 5u * j + 3;
                ok = spin_wait(&v_full[j & 1], (uint32_t)((j >> 1) & 1), abort_flag);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    uint4 *z = reinterpret_cast<uint4 *>(smem + kOffRing + slot_of(blk + i) * kBlockBytes + (tid & 127) * 128);
                    if (ok && (tid & 127) >= there) {
#pragma unroll
                        for (int c = 0; c < 8; c++) z[c] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            tc_fence_before();
            mbar_arrive(&p_full[w]);
        }
        if (ok && nt > 0)
            ok = __all_sync(0xffffffffu,
                            mbar_wait_bounded(&pv_done[w], (uint32_t)((nt - 1) & 1), kWaitLimitE, abort_flag));
        // (a part goes over the ring, which the other query tile's last product may still read)
        if (ok && nt > 0 && C > 1 && nwg > 1)
            ok = __all_sync(0xffffffffu,
                            mbar_wait_bounded(&pv_done[1 - w], (uint32_t)((nt - 1) & 1), kWaitLimitE, abort_flag));
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) flag_error(a.err, kErrTimeout);
        } else if (C > 1) {
            // ---- this CTA's part: FP32 rows over the ring (16-byte chunk c of row r at c ^ (r % 32)), (m, l) over Q
            tc_fence_after();
            const int r = w * kQRows + (tid & 127);
            reinterpret_cast<float2 *>(smem + kOffQ)[r] = make_float2(m_run, l_run);
            float4 *row = reinterpret_cast<float4 *>(smem + kOffRing) + r * 32;
#pragma unroll
            for (int cblk = 0; cblk < 4; cblk++) {
                uint32_t ov[32];
                if (nt > 0) {
                    tc_ld32(tmem + lane_base + colO + 32 * cblk, ov);
                    tc_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e++) ov[e] = 0;
                }
#pragma unroll
                for (int e = 0; e < 8; e++)
                    row[(8 * cblk + e) ^ (r & 31)] =
                        make_float4(__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                                    __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3]));
            }
        } else {
            // ---- O / l -> BF16 row of the output
            tc_fence_after();
            const float inv = 1.f / l_run;
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + (((int64_t)q0 + token) * a.H + head) * kHeadDim);
#pragma unroll
            for (int cblk = 0; cblk < 4; cblk++) {
                uint32_t ov[32];
                tc_ld32(tmem + lane_base + colO + 32 * cblk, ov);
                tc_wait_ld();
                if (row_ok) {
#pragma unroll
                    for (int q4 = 0; q4 < 4; q4++) {
                        uint32_t wv[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const __nv_bfloat162 hv = __floats2bfloat162_rn(
                                __uint_as_float(ov[8 * q4 + 2 * e]) * inv, __uint_as_float(ov[8 * q4 + 2 * e + 1]) * inv);
                            wv[e] = *reinterpret_cast<const uint32_t *>(&hv);
                        }
                        dst[4 * cblk + q4] = make_uint4(wv[0], wv[1], wv[2], wv[3]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tc_dealloc(tmem, kTmemCols);
    if (C > 1) {
        // ---- join the parts: this CTA the rank-th share of the rows, a warp per row, lane l dims 4l .. 4l + 3
        cluster.sync();
        const int nrows = min(kCtaRows, L - row0);
        if (warp < kSoftThreads / 32) {
            for (int r = kCtaRows / C * rank + warp; r < min(nrows, kCtaRows / C * (rank + 1)); r += kSoftThreads / 32) {
                float2 ml = make_float2(kNegInfE, 0.f);
                if (lane < C) ml = cluster.map_shared_rank(reinterpret_cast<float2 *>(smem + kOffQ), lane)[r];
                float mx = ml.x;
#pragma unroll
                for (int x = kMaxSplit / 2; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                mx = __shfl_sync(0xffffffffu, mx, 0);
                const float f = ml.x == kNegInfE ? 0.f : ex2(ml.x - mx);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                float l = 0.f;
                for (int c = 0; c < C; c++) {
                    const float4 v = (cluster.map_shared_rank(reinterpret_cast<float4 *>(smem + kOffRing), c) + r * 32)[lane ^ (r & 31)];
                    const float fc = __shfl_sync(0xffffffffu, f, c);
                    l += fc * __shfl_sync(0xffffffffu, ml.y, c);
                    acc.x += fc * v.x;
                    acc.y += fc * v.y;
                    acc.z += fc * v.z;
                    acc.w += fc * v.w;
                }
                const float inv = 1.f / l;
                const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
                const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
                reinterpret_cast<uint2 *>(a.out + (((int64_t)q0 + row0 + r) * a.H + head) * kHeadDim)[lane] =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
            }
        }
        cluster.sync();   // no CTA leaves while its part may be read
    }
}

// [rows][heads][width] BF16 at `base` (strides in elements) as a 3-D map with 64 x 1 x 128 boxes.
bool make_map(CUtensorMap *map, const void *base, int64_t rows, int heads, int width, int64_t token_stride,
              int64_t head_stride) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kKeys};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_latent_extend(const void *q, const void *k_prefix, const void *v_prefix, int64_t pre_token,
                                 int64_t pre_head, const void *rope_prefix, const int32_t *cu_prefix,
                                 int64_t total_prefix, const void *k_chunk, const void *v_chunk, int64_t new_token,
                                 int64_t new_head, const void *rope_chunk, const int32_t *cu_q, int64_t total_q,
                                 int num_reqs, int max_q_len, int num_heads, float sm_scale, void *out, unsigned *err,
                                 cudaStream_t stream) {
    static std::mutex mu;
    static bool attr_set[64] = {};
    static int waves[64][3];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::unique_lock<std::mutex> lock(mu);
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&latent_extend_kernel),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kESmem);
        if (e != cudaSuccess) return e;
        // clusters of 2, 4 and 8 CTAs that the device holds at once
        for (int k = 0; k < 3; k++) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2u << k);
            cfg.blockDim = dim3(kEThreads);
            cfg.dynamicSmemBytes = kESmem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2u << k;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&waves[dev][k], reinterpret_cast<const void *>(&latent_extend_kernel), &cfg);
            if (e != cudaSuccess) return e;
        }
        attr_set[dev] = true;
    }
    lock.unlock();
    ExtendMaps maps;
    if (!make_map(&maps.k_new, k_chunk, total_q, num_heads, kHeadDim, new_token, new_head) ||
        !make_map(&maps.v_new, v_chunk, total_q, num_heads, kHeadDim, new_token, new_head) ||
        !make_map(&maps.r_new, rope_chunk, total_q, 1, kRopeDim, kRopeDim, kRopeDim))
        return cudaErrorInvalidValue;
    if (total_prefix == 0) {   // never used
        maps.k_pre = maps.k_new;
        maps.v_pre = maps.v_new;
        maps.r_pre = maps.r_new;
    } else if (!make_map(&maps.k_pre, k_prefix, total_prefix, num_heads, kHeadDim, pre_token, pre_head) ||
               !make_map(&maps.v_pre, v_prefix, total_prefix, num_heads, kHeadDim, pre_token, pre_head) ||
               !make_map(&maps.r_pre, rope_prefix, total_prefix, 1, kRopeDim, kRopeDim, kRopeDim)) {
        return cudaErrorInvalidValue;
    }
    ExtendArgs a = {};
    a.q = static_cast<const uint16_t *>(q);
    a.cu_prefix = cu_prefix;
    a.cu_q = cu_q;
    a.H = num_heads;
    a.max_q_len = max_q_len;
    a.total_q = total_q;
    a.total_prefix = total_prefix;
    a.score_log2 = (float)((double)sm_scale * 1.4426950408889634);
    a.out = static_cast<uint16_t *>(out);
    a.err = err;
    const int64_t qtiles = ceil_div64(max_q_len, kCtaRows), ctas = qtiles * num_heads * num_reqs;
    const int64_t tiles = (total_prefix + (total_q < (int64_t)num_reqs * max_q_len ? total_q : (int64_t)num_reqs * max_q_len)) /
                          num_reqs / kKeys;   // K/V tiles of an average request
    // Clusters share the K/V tiles of a CTA while the grid stays one wave of them: 32 heads x 2
    // query tiles of one request over 8,192 tokens take 148 us as 64 CTAs and 88 us as 64
    // clusters of two (157 us as 64 of four, which are two waves); 256 CTAs that are two waves
    // already take the same either way.  A tile a CTA is enough (8 heads, 64 queries over 1,100 tokens:
    // 15.8 us in clusters of eight, 18.5 of four, 22.0 of two; over 300 tokens 16.7 of two, 15.5 alone).
    int split = 1;
    for (int k = 0; k < 3; k++)
        if (ctas <= waves[dev][k] && tiles >= (kMinTiles > (2 << k) ? kMinTiles : 2 << k)) split = 2 << k;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(qtiles * split), (unsigned)num_heads, (unsigned)num_reqs);
    cfg.blockDim = dim3(kEThreads);
    cfg.dynamicSmemBytes = kESmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void *args[] = {&maps, &a};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(&latent_extend_kernel), args);
}

}  // namespace nvfp4kv
