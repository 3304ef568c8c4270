// attention_weights.cu -- the attention weight of every cached token, added to its score.
//
//   scores[b][h][t] += sum_j softmax_t(sm_scale * g_K * q_j . k_t)[t]
// over the G query heads j of kv head h: what a policy that evicts tokens by
// accumulated attention weight keeps.  K alone is needed (72 of a token's 144
// NVFP4 bytes), but the softmax's denominators are known only after all of a
// sequence, and the weights are held in FP32 (decode rounds its
// probabilities to FP16, which a running sum would keep).
//
// Two kernels walk the same flat order of 96-token units (sequence, kv head,
// unit), cut into one contiguous piece a warp:
//   stats    running maximum and sum of 2^(s - m), kept by every thread for its
//            own (token, head) positions and joined only where the warp leaves a
//            (sequence, head) pair: one (m, l) partial per warp, pair and head;
//   weights  joins the partials of a pair into L = m + log2 l, forms the scores'
//            products again and adds sum_j 2^(s_j - L_j): no atomics, one
//            addition per entry.
// Every warp has two 96-token stages that it fills itself with bulk copies of the
// groups' K halves, a unit ahead (loads to registers left the warps waiting for
// memory a third of the time, and held 36 registers; three stages of 64 tokens: 105
// us for the case below, two 104, two of 80 tokens 102, two of 96 101).  The
// scores come from mma.sync m16n8k16 with the 16 tokens of a group on M and the
// heads on N.  The contraction's order is free, so thread j of a quad takes the
// dimensions 32j .. 32j + 31 of its tokens: 16 contiguous bytes of codes a token;
// e2m1 x e4m3 is an exact FP16 value, and q is FP16 after a power-of-two pre-scale a head
// (exact above 2^-29 of its largest value), undone in the FP32 score factor.
//
// 16 sequences of up to 32,768 tokens, 64 query and 8 kv heads: 94 us (stats 45, the
// rest weights), of which one reading of K is 32 us.  Each pass is bound by unpacking: some 160
// instructions a 16-token group, half of the ALU's slots, at four warps a scheduler.
// Three CTAs an SM (80 registers, 64-token units) took 122 us.
#include <mutex>

#include "common.cuh"
#include "flat_plan.cuh"
#include "kernels.h"
#include "quantize.cuh"

namespace nvfp4kv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarpsW = kThreads / 32;
constexpr int kUnit = kScoreUnit;                     // tokens per unit
constexpr int kGroupsW = kUnit / 16;
constexpr int kStagesW = 2;                   // ring stages of a warp
constexpr uint32_t kWaitLimitW = 1u << 24;
constexpr float kNegInfW = -__builtin_huge_valf();

template <int DTYPE>
struct KHalf {   // a group's K bytes: NVFP4 codes [16][64] and scales [16][8], or FP8 [16][128]
    static constexpr int kGroup = DTYPE == NVFP4KV_DTYPE_NVFP4 ? 2304 : 4096;
    static constexpr int kBytes = DTYPE == NVFP4KV_DTYPE_NVFP4 ? 1152 : 2048;
    static constexpr int kStage = kGroupsW * kBytes;
    static constexpr int kSmem = kWarpsW * kStagesW * kStage;
};

struct WeightsArgs {
    const uint8_t *pool;
    int64_t num_pages;
    int P, log2P, Hkv, G, Hq, B, max_pages;
    int64_t slab;
    const uint16_t *q;
    const int32_t *block_table, *seq_lens;
    int64_t cap;            // rows a sequence may have: min(table, score_stride)
    float score_log2;       // sm_scale * g_K * log2(e)
    float *scores;
    int64_t score_stride;
    float2 *part;           // [workers + B * Hkv][G]: (m, l) of warp w and pair p at w + p
    int workers;
    unsigned *err;
};

// Scores (before the factor) of 16 tokens whose K half lies at k: c[x] = rows g, g + 8 x heads 8 x + 2j, + 1.
template <int DTYPE, int NT>
__device__ __forceinline__ void group_scores(const uint8_t *k, int lane, const uint32_t (&qf)[NT][16], float (&c)[NT][4]) {
    const int g = lane >> 2, j = lane & 3;
#pragma unroll
    for (int x = 0; x < NT; x++) c[x][0] = c[x][1] = c[x][2] = c[x][3] = 0.f;
    uint32_t f[2][16];   // token g / g + 8: f16 pairs of dimensions 32j + 2p, + 1
#pragma unroll
    for (int e = 0; e < 2; e++) {
        const int row = g + 8 * e;
        if (DTYPE == NVFP4KV_DTYPE_NVFP4) {
            const uint4 w = *reinterpret_cast<const uint4 *>(k + row * 64 + j * 16);
            e2m1x8_to_f16x2x4(w.x, f[e][0], f[e][1], f[e][2], f[e][3]);
            e2m1x8_to_f16x2x4(w.y, f[e][4], f[e][5], f[e][6], f[e][7]);
            e2m1x8_to_f16x2x4(w.z, f[e][8], f[e][9], f[e][10], f[e][11]);
            e2m1x8_to_f16x2x4(w.w, f[e][12], f[e][13], f[e][14], f[e][15]);
            const uint32_t s2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(k + 1024 + row * 8 + j * 2));
            const uint32_t lo = __byte_perm(s2, s2, 0x1010), hi = __byte_perm(s2, s2, 0x3232);
#pragma unroll
            for (int p = 0; p < 8; p++) {
                f[e][p] = hmul2(f[e][p], lo);
                f[e][8 + p] = hmul2(f[e][8 + p], hi);
            }
        } else {
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const uint4 v = *reinterpret_cast<const uint4 *>(k + row * 128 + j * 32 + x * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    f[e][8 * x + 2 * p] = e4m3x2_to_f16x2(w[p] & 0xffffu);
                    f[e][8 * x + 2 * p + 1] = e4m3x2_to_f16x2(w[p] >> 16);
                }
            }
        }
    }
#pragma unroll
    for (int s = 0; s < 8; s++)
#pragma unroll
        for (int x = 0; x < NT; x++)
            mma_f16_16816(c[x], f[0][2 * s], f[1][2 * s], f[0][2 * s + 1], f[1][2 * s + 1], qf[x][2 * s], qf[x][2 * s + 1]);
}

// This thread's query fragments (heads 8 x + lane / 4, dimensions 32 (lane % 4) ..)
// and the score factors of heads 8 x + 2 (lane % 4), + 1.
template <int NT>
__device__ __forceinline__ void load_query(const WeightsArgs &a, int b, int h, int lane, uint32_t (&qf)[NT][16],
                                           float (&fac)[NT][2]) {
    const int j = lane & 3;
#pragma unroll
    for (int x = 0; x < NT; x++) {
        const int head = 8 * x + (lane >> 2);
        uint32_t w[16], m = 0;
        if (head < a.G) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                a.q + ((int64_t)b * a.Hq + (int64_t)h * a.G + head) * kHeadDim + 32 * j);
#pragma unroll
            for (int p = 0; p < 4; p++) {
                const uint4 v = __ldg(src + p);
                w[4 * p] = v.x;
                w[4 * p + 1] = v.y;
                w[4 * p + 2] = v.z;
                w[4 * p + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int p = 0; p < 16; p++) w[p] = 0;
        }
#pragma unroll
        for (int p = 0; p < 16; p++) m = max_u16x2(m, w[p] & 0x7fff7fffu);
        m = max(m >> 16, m & 0xffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int kq = m ? min(126, max(-126, 14 - ((int)(m >> 7) - 127))) : 0;   // largest |q| into [2^14, 2^15)
        const float sc = __uint_as_float((uint32_t)(kq + 127) << 23);
#pragma unroll
        for (int p = 0; p < 16; p++) qf[x][p] = f32x2_to_f16x2(bf16_hi(w[p]) * sc, bf16_lo(w[p]) * sc);
        const float f = a.score_log2 * __uint_as_float((uint32_t)(127 - kq) << 23);
        fac[x][0] = __shfl_sync(0xffffffffu, f, 8 * j);
        fac[x][1] = __shfl_sync(0xffffffffu, f, 8 * j + 4);
    }
}

// A warp's units in order.
struct UnitIter {
    int b, h, t, n;   // sequence, kv head, first token, the sequence's rows
    int left;         // units of the piece from this one on
};

__device__ __forceinline__ void next_unit(const WeightsArgs &a, UnitIter &it) {
    it.left--;
    it.t += kUnit;
    if (it.t < it.n) return;
    it.t = 0;
    if (++it.h < a.Hkv || it.left <= 0) return;
    it.h = 0;
    do {              // left > 0: a later sequence has units
        it.b++;
        it.n = clamp_rows(__ldg(a.seq_lens + it.b), a.cap);
    } while (it.n == 0);
}

// Page of the unit's lane-th group (lanes 0 .. kGroupsW - 1).
__device__ __forceinline__ int32_t unit_page(const WeightsArgs &a, const UnitIter &it, int lane) {
    const int t = it.t + 16 * lane;
    if (lane >= kGroupsW || it.left <= 0 || t >= it.n) return -1;
    return __ldg(a.block_table + (int64_t)it.b * a.max_pages + (t >> a.log2P));
}

template <int DTYPE, int NT, bool kStats>
__global__ void __launch_bounds__(kThreads, 2) weights_kernel(WeightsArgs a) {
    using H = KHalf<DTYPE>;
    extern __shared__ __align__(128) uint8_t ring_all[];   // [warp][stage][group]
    __shared__ FlatScratch<kThreads> scratch;
    __shared__ uint64_t bars[kWarpsW][kStagesW];
    __shared__ int abort_all;
    // Lengths, q, the cache and the scores may come from earlier work, which is done when the stats
    // kernel has passed its wait: it lets the weights kernel start only then, and that one has to
    // wait again for the partials alone (2 x 300 tokens: 11.1 us, 9.3 so;
    // 16 x 32,768: 99 and 94).
    if (kStats) {
        pdl_wait();
        pdl_launch_dependents();
    }
    const int lane = threadIdx.x & 31;
    const unsigned worker = blockIdx.x * kWarpsW + (threadIdx.x >> 5);
    auto rows = [&](int b) { return clamp_rows(__ldg(a.seq_lens + b), a.cap); };
    auto units = [&](int b) { return (rows(b) + kUnit - 1) / kUnit; };
    if (kStats && blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += kThreads) {
            const int32_t n = a.seq_lens[b];
            if (n < 0 || (int64_t)n > a.cap) flag_error(a.err, kErrSeqLen);
        }
    int b;
    unsigned first, u0 = 0, u1 = 0;
    const unsigned total = flat_locate<kThreads>(
        scratch, a.B, [&](int x) { return a.Hkv * units(x); },
        [&](unsigned t) {
            const FlatCut cut(t, a.workers);
            u0 = cut.begin(worker);
            u1 = cut.begin(worker + 1);
            return u0 < u1 ? u0 : kFlatNone;
        },
        b, first);
    if (threadIdx.x == 0) abort_all = 0;
    __syncthreads();
    if (u0 >= u1) {         // more warps than units
        pdl_wait();         // (no CTA of the weights kernel ends before the stats kernel has)
        return;
    }
    UnitIter it;
    it.b = b;
    it.n = rows(b);
    const int nu0 = units(b);
    it.h = (int)((u0 - first) / (unsigned)nu0);
    it.t = (int)((u0 - first) % (unsigned)nu0) * kUnit;
    it.left = (int)(u1 - u0);
    uint32_t qf[NT][16];
    float fac[NT][2], m[NT][2], l[NT][2];   // kStats: running maximum and sum; else m = L of the pair's heads
    bool fresh = true;
    unsigned u = u0;                        // position in the flat order
    // The warp's ring: unit i of the piece into stage i % kStagesW, requested kStagesW - 1 units
    // ahead (its pages one unit earlier still).
    uint8_t *ring = ring_all + (threadIdx.x >> 5) * (kStagesW * H::kStage);
    uint64_t *bar = bars[threadIdx.x >> 5];
    const volatile int *abort_flag = &abort_all;
    if (lane == 0) {
        for (int i = 0; i < kStagesW; i++) mbar_init(&bar[i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    auto request = [&](const UnitIter &x, int32_t page, int stage) {   // lane i < kGroupsW: group i
        uint8_t *dst = ring + stage * H::kStage + lane * H::kBytes;
        const int t = x.t + 16 * lane;
        bool copy = x.left > 0 && lane < kGroupsW && t < x.n;
        if (copy && (page < 0 || page >= a.num_pages)) {   // reads as zeros
            flag_error(a.err, kErrPage);
            for (int i = 0; i < H::kBytes / 16; i++) reinterpret_cast<uint4 *>(dst)[i] = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before a later unit's copy to the same place
            copy = false;
        }
        const unsigned copies = __popc(__ballot_sync(0xffffffffu, copy));
        if (lane == 0) mbar_arrive_expect_tx(&bar[stage], copies * H::kBytes);
        __syncwarp();
        if (copy)
            bulk_g2s(dst, a.pool + ((int64_t)page * a.Hkv + x.h) * a.slab + ((t & (a.P - 1)) >> 4) * H::kGroup, H::kBytes,
                     &bar[stage]);
    };
    UnitIter nx = it;
    int32_t npage = unit_page(a, nx, lane);
#pragma unroll
    for (int i = 0; i < kStagesW - 1; i++) {
        if (nx.left <= 0) break;
        request(nx, npage, i);
        next_unit(a, nx);
        npage = unit_page(a, nx, lane);
    }
    int stage = 0, ahead = kStagesW - 1;
    uint32_t parity = 0;
    bool ok = true;
    for (; it.left > 0; u++) {
        if (nx.left > 0) {   // into the stage of the unit before this one, which the whole warp has read
            __syncwarp();
            request(nx, npage, ahead);
            next_unit(a, nx);
            npage = unit_page(a, nx, lane);
        }
        if (++ahead == kStagesW) ahead = 0;
        const bool fast = it.t + kUnit <= it.n;   // a whole unit: no masks
        b = it.b;
        const int h = it.h, n = it.n, t0 = it.t;
        const int g = lane >> 2, j = lane & 3;
        float *dst = a.scores + ((int64_t)b * a.Hkv + h) * a.score_stride + t0 + g + 8 * (j & 1);
        float old[kGroupsW];
        if (!kStats) {   // lanes j = 0 and 1 of a quad own tokens g and g + 8
#pragma unroll
            for (int i = 0; i < kGroupsW; i++) {
                old[i] = 0.f;
                if (j < 2 && (fast || t0 + 16 * i + g + 8 * j < n)) old[i] = dst[16 * i];
            }
        }
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar[stage], parity, kWaitLimitW, abort_flag));
        if (!ok) break;
        const uint8_t *unit = ring + stage * H::kStage;
        if (++stage == kStagesW) {
            stage = 0;
            parity ^= 1;
        }
        if (fresh) {
            load_query<NT>(a, b, h, lane, qf, fac);
            if (kStats) {
#pragma unroll
                for (int x = 0; x < NT; x++) {
                    m[x][0] = m[x][1] = kNegInfW;
                    l[x][0] = l[x][1] = 0.f;
                }
            } else {
                pdl_wait();
                // the pair's units [p0, p0 + nu) were covered by these warps
                const int nu = (n + kUnit - 1) / kUnit;
                const FlatCut cut(total, a.workers);
                const int64_t p = (int64_t)b * a.Hkv + h;
                const unsigned p0 = u - t0 / kUnit, w0 = cut.piece(p0), w1 = cut.piece(p0 + nu - 1);
                float mine[NT * 8];
#pragma unroll
                for (int hd = 0; hd < NT * 8; hd++) {
                    mine[hd] = -kNegInfW;      // heads that do not exist: weight 2^-inf
                    if (hd >= a.G) continue;   // uniform
                    float mm = kNegInfW, ll = 0.f;
                    for (unsigned w = w0 + lane; w <= w1; w += 32) {
                        const float2 v = __ldcg(a.part + (w + p) * a.G + hd);
                        const float mx = fmaxf(mm, v.x);
                        if (mx != kNegInfW) ll = ll * ex2(mm - mx) + v.y * ex2(v.x - mx);
                        mm = mx;
                    }
#pragma unroll
                    for (int x = 16; x; x >>= 1) {
                        const float om = __shfl_xor_sync(0xffffffffu, mm, x), ol = __shfl_xor_sync(0xffffffffu, ll, x);
                        const float mx = fmaxf(mm, om);
                        if (mx != kNegInfW) ll = ll * ex2(mm - mx) + ol * ex2(om - mx);
                        mm = mx;
                    }
                    mine[hd] = mm + __log2f(ll);
                }
#pragma unroll
                for (int x = 0; x < NT; x++) {
                    m[x][0] = m[x][1] = 0.f;
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        if ((lane & 3) == q) {
                            m[x][0] = mine[8 * x + 2 * q];
                            m[x][1] = mine[8 * x + 2 * q + 1];
                        }
                }
            }
        }
        float sc[kStats ? kGroupsW : 1][NT][4];
#pragma unroll
        for (int i = 0; i < kGroupsW; i++) {
            float c[NT][4];
            group_scores<DTYPE, NT>(unit + i * H::kBytes, lane, qf, c);
            const bool ok0 = fast || t0 + 16 * i + g < n, ok1 = fast || t0 + 16 * i + g + 8 < n;
            if (kStats) {
#pragma unroll
                for (int x = 0; x < NT; x++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        sc[kStats ? i : 0][x][e] = (e < 2 ? ok0 : ok1) ? c[x][e] * fac[x][e & 1] : kNegInfW;
            } else {
                float w0 = 0.f, w1 = 0.f;
#pragma unroll
                for (int x = 0; x < NT; x++) {
                    w0 += ex2(fmaf(c[x][0], fac[x][0], -m[x][0])) + ex2(fmaf(c[x][1], fac[x][1], -m[x][1]));
                    w1 += ex2(fmaf(c[x][2], fac[x][0], -m[x][0])) + ex2(fmaf(c[x][3], fac[x][1], -m[x][1]));
                }
                w0 += __shfl_xor_sync(0xffffffffu, w0, 1);
                w1 += __shfl_xor_sync(0xffffffffu, w1, 1);
                w0 += __shfl_xor_sync(0xffffffffu, w0, 2);
                w1 += __shfl_xor_sync(0xffffffffu, w1, 2);
                if (j < 2 && (j ? ok1 : ok0)) dst[16 * i] = old[i] + (j ? w1 : w0);
            }
        }
        if (kStats) {
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float mx = m[x][e];
#pragma unroll
                    for (int i = 0; i < kGroupsW; i++)
                        mx = fmaxf(mx, fmaxf(sc[kStats ? i : 0][x][e], sc[kStats ? i : 0][x][e + 2]));
                    if (mx != kNegInfW) {
                        float s = l[x][e] * ex2(m[x][e] - mx);
#pragma unroll
                        for (int i = 0; i < kGroupsW; i++)
                            s += ex2(sc[kStats ? i : 0][x][e] - mx) + ex2(sc[kStats ? i : 0][x][e + 2] - mx);
                        l[x][e] = s;
                        m[x][e] = mx;
                    }
                }
        }
        next_unit(a, it);
        fresh = it.left <= 0 || it.b != b || it.h != h;
        if (kStats && fresh) {   // this warp's partial of the pair: join the eight token rows of each head
            const int64_t at = (worker + (int64_t)b * a.Hkv + h) * a.G;
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float mm = m[x][e], ll = l[x][e];
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) {
                        const float om = __shfl_xor_sync(0xffffffffu, mm, s), ol = __shfl_xor_sync(0xffffffffu, ll, s);
                        const float mx = fmaxf(mm, om);
                        if (mx != kNegInfW) ll = ll * ex2(mm - mx) + ol * ex2(om - mx);
                        mm = mx;
                    }
                    const int hd = 8 * x + 2 * j + e;
                    if (g == 0 && hd < a.G) a.part[at + hd] = make_float2(mm, ll);
                }
        }
    }
    if (!ok) {   // no copy may still be writing when the CTA's memory is freed: units [it, nx) were requested
        abort_all = 1;
        if (lane == 0) flag_error(a.err, kErrTimeout);
        for (; it.left > nx.left; it.left--) {
            mbar_wait_bounded(&bar[stage], parity, kWaitLimitW, nullptr);
            if (++stage == kStagesW) {
                stage = 0;
                parity ^= 1;
            }
        }
    }
}

template <bool kStats>
const void *weights_fn(int dtype, int nt) {
    if (dtype == NVFP4KV_DTYPE_NVFP4)
        return nt == 1 ? reinterpret_cast<const void *>(&weights_kernel<0, 1, kStats>)
                       : reinterpret_cast<const void *>(&weights_kernel<0, 2, kStats>);
    return nt == 1 ? reinterpret_cast<const void *>(&weights_kernel<1, 1, kStats>)
                   : reinterpret_cast<const void *>(&weights_kernel<1, 2, kStats>);
}

int weights_smem(int dtype) { return dtype == NVFP4KV_DTYPE_NVFP4 ? KHalf<0>::kSmem : KHalf<1>::kSmem; }

constexpr int kMaxDevicesW = 64;
std::mutex g_mu_w;
int g_workers[kMaxDevicesW][2][2];

}  // namespace

int weights_workers(int dtype, int group, cudaError_t *status) {
    const int nt = group <= 8 ? 1 : 2;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevicesW)) e = cudaErrorInvalidDevice;
    int out = 0;
    if (e == cudaSuccess) {
        std::lock_guard<std::mutex> lock(g_mu_w);
        int &w = g_workers[dev][dtype][nt - 1];
        if (!w) {
            int sms = 0, a = 0, b = 0;
            const int smem = weights_smem(dtype);
            const void *fa = weights_fn<true>(dtype, nt), *fb = weights_fn<false>(dtype, nt);
            e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(fa, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(fb, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&a, fa, kThreads, smem);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, fb, kThreads, smem);
            if (e == cudaSuccess) w = sms * (a < b ? (a > 0 ? a : 1) : (b > 0 ? b : 1)) * kWarpsW;
        }
        out = w;
    }
    if (status) *status = e;
    return e == cudaSuccess ? out : 0;
}

size_t weights_workspace_bytes(int batch, int num_q_heads, int num_kv_heads, int workers) {
    return ((size_t)workers + (size_t)batch * num_kv_heads) * (num_q_heads / num_kv_heads) * sizeof(float2);
}

cudaError_t launch_weights(const nvfp4kv_cache &c, const void *q, int batch, int num_q_heads,
                           const int32_t *block_table, int max_pages, const int32_t *seq_lens, float sm_scale,
                           float *scores, int64_t score_stride, void *workspace, int workers, unsigned *err,
                           cudaStream_t stream) {
    WeightsArgs a;
    a.pool = static_cast<const uint8_t *>(c.pool);
    a.num_pages = c.num_pages;
    a.P = c.page_size;
    a.log2P = __builtin_ctz((unsigned)c.page_size);
    a.Hkv = c.num_kv_heads;
    a.G = num_q_heads / c.num_kv_heads;
    a.Hq = num_q_heads;
    a.B = batch;
    a.max_pages = max_pages;
    a.slab = (int64_t)(c.dtype == NVFP4KV_DTYPE_NVFP4 ? 144 : 256) * c.page_size;
    a.q = static_cast<const uint16_t *>(q);
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    const int64_t table = (int64_t)max_pages * c.page_size;
    a.cap = table < score_stride ? table : score_stride;
    a.score_log2 = (float)((double)sm_scale * (double)c.k_global_scale * 1.4426950408889634);
    a.scores = scores;
    a.score_stride = score_stride;
    a.part = static_cast<float2 *>(workspace);
    a.workers = workers;
    a.err = err;
    const int nt = a.G <= 8 ? 1 : 2;
    void *args[] = {&a};
    cudaError_t e = launch_pdl(weights_fn<true>(c.dtype, nt), (unsigned)(workers / kWarpsW), kThreads, (size_t)weights_smem(c.dtype), stream, args);
    if (e != cudaSuccess) return e;
    return launch_pdl(weights_fn<false>(c.dtype, nt), (unsigned)(workers / kWarpsW), kThreads, (size_t)weights_smem(c.dtype), stream, args);
}

}  // namespace nvfp4kv
