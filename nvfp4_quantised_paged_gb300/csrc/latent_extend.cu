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
// thread; one thread of warp 8 drives the TMA loads and the tcgen05 products, two
// independent chains that the tensor core overlaps.  What differs:
//   * S_w = Q_w K^T takes twelve K 16 steps, eight over K's two column blocks and
//     four over the rotary block, a third column block of the K slot that its own
//     tensor map fills: 48 KB a K slot and a query tile;
//   * Q 96 KB + two K slots 96 KB leave room for one V slot (32 KB): V(j + 1) is
//     requested when both O_w += P_w(j) V(j) are done, and is needed only after
//     S(j + 1) and its softmax, so one slot costs little where one K slot would
//     put every K load on the critical path;
//   * rows of a V tile past the request's end are zeroed in shared memory before
//     the product: they are other requests' rows or padding, and a NaN there times
//     a probability of 0 would still be a NaN.
// Bound by the tensor cores: 2 * (192 + 128) flops a (query, key, head), K and V
// tiles shared by 256 queries through L2.  Every wait is bounded.
#include "common.cuh"
#include "extend_common.cuh"
#include "kernels.h"
#include "latent.cuh"
#include "tcgen05.cuh"

namespace nvfp4kv {

namespace {

constexpr int kWGs = 2;
constexpr int kQRows = 128;
constexpr int kCtaRows = kWGs * kQRows;
constexpr int kSoftThreads = kWGs * kQRows;
constexpr int kEThreads = kSoftThreads + 32;   // + the load / MMA warp
constexpr int kKeys = 128;
constexpr int kQkDim = kHeadDim + kRopeDim;    // 192
constexpr int kBlockBytes = 128 * 128;         // one column block: 128 rows of 64 BF16 values
constexpr int kQBytes = 3 * kBlockBytes, kKTile = 3 * kBlockBytes, kVTile = 2 * kBlockBytes;
constexpr int kOffQ = 0;
constexpr int kOffK = kWGs * kQBytes;          // K slots [2]
constexpr int kOffV = kOffK + 2 * kKTile;      // one V slot
constexpr int kOffBar = kOffV + kVTile;
constexpr int kNumBars = 10;                   // k_full[2] v_full s_done[2] p_full[2] pv_done[2] drain
constexpr int kOffTmem = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kOffOrder = kOffBar + 256;       // int[256]: requests by decreasing prefix length
constexpr int kOrderMax = 256;
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

// K/V as 3-D maps [rows][heads][128] (any strides), the rotary rows as [rows][1][64]; boxes of 64 x 1 x 128.
struct ExtendMaps {
    CUtensorMap k_pre, v_pre, r_pre, k_new, v_new, r_new;
};

__global__ void __launch_bounds__(kEThreads, 1)
    latent_extend_kernel(const __grid_constant__ ExtendMaps maps, ExtendArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *k_full = bars, *v_full = bars + 2, *s_done = bars + 3, *p_full = bars + 5, *pv_done = bars + 7;
    uint64_t *drain = bars + 9;
    uint32_t &tmem_base = *reinterpret_cast<uint32_t *>(smem + kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffAbort);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    const int row0 = blockIdx.x * kCtaRows;
    if (row0 >= L) return;
    const int nwg = row0 + kQRows < L ? 2 : 1;                  // query tiles holding rows
    const int t_last = min(row0 + kCtaRows, L) - 1;             // last chunk token of this CTA
    const int nt_pre = (np + kKeys - 1) / kKeys;
    const int nt = nt_pre + t_last / kKeys + 1;
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
    auto load_k = [&](int j) {
        const bool pre = j < nt_pre;
        const uint32_t dst = sbase + kOffK + (j & 1) * kKTile;
        mbar_arrive_expect_tx(&k_full[j & 1], kKTile);
        tma_load_3d(dst, pre ? &maps.k_pre : &maps.k_new, 0, head, tile_row(j), &k_full[j & 1]);
        tma_load_3d(dst + kBlockBytes, pre ? &maps.k_pre : &maps.k_new, 64, head, tile_row(j), &k_full[j & 1]);
        tma_load_3d(dst + 2 * kBlockBytes, pre ? &maps.r_pre : &maps.r_new, 0, 0, tile_row(j), &k_full[j & 1]);
    };
    auto load_v = [&](int j) {
        const CUtensorMap *m = j < nt_pre ? &maps.v_pre : &maps.v_new;
        mbar_arrive_expect_tx(v_full, kVTile);
        tma_load_3d(sbase + kOffV, m, 0, head, tile_row(j), v_full);
        tma_load_3d(sbase + kOffV + kBlockBytes, m, 64, head, tile_row(j), v_full);
    };

    if (warp == 0) tc_alloc(&tmem_base, kTmemCols);
    if (tid == kSoftThreads) {
        for (int j = 0; j < kNumBars; j++) mbar_init(&bars[j], j == 5 || j == 6 ? kQRows : 1);
        *abort_flag = 0;
        fence_mbar_init();
        load_k(0);
        load_v(0);
        if (nt > 1) load_k(1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // Q for the tensor core
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;

    if (warp == kSoftThreads / 32) {
        // ---------------- load / MMA warp: the whole warp runs the loop and one elected lane
        // issues, so that descriptors stay uniform values (issued under a divergent branch a
        // product cost more than the tensor core's 64 clocks for it)
        {
            constexpr uint32_t idesc_s = idesc_bf16_f32(128, kKeys, false);
            constexpr uint32_t idesc_o = idesc_bf16_f32(128, kHeadDim, true);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const bool leader = elect_one();
            const uint64_t dQ = smem_desc_sw128(sbase + kOffQ, 16, 1024), dK = smem_desc_sw128(sbase + kOffK, 16, 1024);
            const uint64_t dV = smem_desc_sw128(sbase + kOffV, kBlockBytes, 1024);
            auto mma_s = [&](uint32_t w, uint32_t s) {  // S_w = Q_w K(slot s)^T over 192 dimensions, 16 at a time
                const uint64_t q = dQ + w * (kQBytes / 16), k = dK + s * (kKTile / 16);
#pragma unroll
                for (int kk = 0; kk < 12; kk++) {
                    const uint32_t off = (uint32_t)(kk >> 2) * (kBlockBytes / 16) + (uint32_t)(kk & 3) * 2;
                    tc_mma_bf16(tm + 128u * w, q + off, k + off, idesc_s, kk > 0);
                }
                tc_commit(&s_done[w]);
            };
            auto mma_pv = [&](uint32_t w, int j) {  // O_w += P_w V over the tile's 128 keys
                const uint32_t acc = j > 0 ? 1u : 0u;
#pragma unroll
                for (int kk = 0; kk < 8; kk++)  // P from TMEM: 8 columns = 16 keys
                    tc_mma_bf16_tmem_a(tm + kColO + 128u * w, tm + 128u * w + kk * 8, dV + kk * 128, idesc_o,
                                       kk > 0 ? 1u : acc);
                tc_commit(&pv_done[w]);
            };
            // Issue whatever is ready, for either query tile (the order of extend_attention.cu):
            //   S_w(t) once K(t) has landed and O_w += P_w(t - 1) V(t - 1) is complete;
            //   O_w += P_w(t) V(t) once P_w(t) is stored (and, so, V(t) has landed: its threads waited for it);
            //   K(t) into slot t % 2 once both S(t - 2) are done (their P V issued);
            //   V(t) once both P(t - 1) V(t - 1) are complete.
            int tw[kWGs] = {0, 0};
            bool at_pv[kWGs] = {false, false};
            int pv_seen[kWGs] = {0, 0};
            int k_next = nt > 1 ? 2 : 1, v_next = 1;
            bool ok = true;
            uint32_t idle = 0;
            for (;;) {
                bool progress = false, finished = true;
#pragma unroll
                for (int w = 0; w < kWGs; w++) {
                    const int t = tw[w];
                    if (w >= nwg || t >= nt) continue;
                    finished = false;
                    if (!at_pv[w]) {
                        if (t > 0 && pv_seen[w] < t) {
                            if (!__all_sync(0xffffffffu, mbar_test_wait(&pv_done[w], (uint32_t)((t - 1) & 1)))) continue;
                            pv_seen[w] = t;
                            progress = true;
                        }
                        if (!__all_sync(0xffffffffu, mbar_test_wait(&k_full[t & 1], (uint32_t)((t >> 1) & 1)))) continue;
                        tc_fence_after();
                        if (leader) mma_s(w, t & 1);
                        at_pv[w] = true;
                    } else {
                        if (!__all_sync(0xffffffffu, mbar_test_wait(&p_full[w], (uint32_t)(t & 1)))) continue;
                        tc_fence_after();
                        if (leader) mma_pv(w, t);
                        at_pv[w] = false;
                        tw[w] = t + 1;
                    }
                    progress = true;
                }
                if (finished) break;
                int min_tw = tw[0], min_seen = pv_seen[0];
                if (nwg > 1) {
                    min_tw = min(min_tw, tw[1]);
                    min_seen = min(min_seen, pv_seen[1]);
                }
                if (k_next < nt && min_tw >= k_next - 1) {
                    if (leader) load_k(k_next);
                    k_next++;
                    progress = true;
                }
                if (v_next < nt && min_seen >= v_next) {
                    if (leader) load_v(v_next);
                    v_next++;
                    progress = true;
                }
                if (progress) {
                    idle = 0;
                } else if (++idle > kWaitLimitE || __any_sync(0xffffffffu, *abort_flag)) {
                    ok = false;
                    break;
                }
            }
            if (!ok && leader) {
                *abort_flag = 1;
                flag_error(a.err, kErrTimeout);
                // no copy or product may still be running when the CTA frees its memory
                for (int t = max(0, k_next - 2); t < k_next; t++)
                    mbar_wait_bounded(&k_full[t & 1], (uint32_t)((t >> 1) & 1), kWaitLimitE, nullptr);
                mbar_wait_bounded(v_full, (uint32_t)((v_next - 1) & 1), kWaitLimitE, nullptr);
                tc_commit(drain);
                mbar_wait_bounded(drain, 0, kWaitLimitE, nullptr);
            }
        }
        __syncwarp();
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
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_done[w], (uint32_t)(j & 1), kWaitLimitE, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const bool pre = j < nt_pre;
            const int base = pre ? j * kKeys : (j - nt_pre) * kKeys;
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
            uint32_t pw0[32], pw1[32];
            float ls[4] = {0.f, 0.f, 0.f, 0.f};
            float smax;
            {
                float sc[64];
                load_half(0, sc);
                smax = half_max(sc);
                make_p(sc, -m_run, pw0, ls);
                load_half(1, sc);
                smax = fmaxf(smax, half_max(sc));
                const float mx = smax * a.score_log2;  // the scale is positive
                const bool need = mx > m_run + kRescale;
                if (!__any_sync(0xffffffffu, need)) {
                    make_p(sc, -m_run, pw1, ls);
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
                    make_p(sc, -m_run, pw1, ls);
                    load_half(0, sc);
                    make_p(sc, -m_run, pw0, ls);
                }
            }
            l_run += (ls[0] + ls[1]) + (ls[2] + ls[3]);
            tc_st32(tmem + lane_base + colS, pw0);       // over scores 0 .. 31 (read already)
            tc_st32(tmem + lane_base + colS + 32, pw1);  // over scores 32 .. 63
            tc_wait_st();
            // V(j) has landed; rows past the request's end (edge tiles only) become zeros.  Both
            // warpgroups write them, each before its own product.
            ok = __all_sync(0xffffffffu, spin_wait(v_full, (uint32_t)(j & 1), abort_flag));
            if (!ok) break;
            const int there = (pre ? np : L) - base;   // rows of the tile that belong to the request
            if (there < kKeys) {
                if ((tid & 127) >= there) {
                    uint4 *z = reinterpret_cast<uint4 *>(smem + kOffV + (tid & 127) * 128);
#pragma unroll
                    for (int c = 0; c < 8; c++) {
                        z[c] = make_uint4(0u, 0u, 0u, 0u);
                        z[kBlockBytes / 16 + c] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            tc_fence_before();
            mbar_arrive(&p_full[w]);
        }
        if (ok)
            ok = __all_sync(0xffffffffu,
                            mbar_wait_bounded(&pv_done[w], (uint32_t)((nt - 1) & 1), kWaitLimitE, abort_flag));
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) flag_error(a.err, kErrTimeout);
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
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&latent_extend_kernel),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kESmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
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
    dim3 grid((unsigned)ceil_div64(max_q_len, kCtaRows), (unsigned)num_heads, (unsigned)num_reqs);
    latent_extend_kernel<<<grid, kEThreads, kESmem, stream>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace nvfp4kv
