// evict.cu -- the tokens of largest score of every sequence and kv head, moved into new pages.
//
// Two kernels:
//   select   one cluster of C CTAs per (sequence, kv head).  With n > keep rows
//            the smallest kept key is found by a radix select over the scores'
//            order-preserving 32-bit keys, 8 bits a round: each CTA counts its
//            part of the rows in shared memory, the cluster adds the 256 counts
//            up through distributed shared memory and every CTA picks the same
//            digit.  Rows that must stay (the first `sink`, the last `recent`)
//            have the largest key; ties at the border go to the lowest index.
//            Then the kept indices are written in order: each warp counts and
//            later compacts a contiguous part of the rows, its offset coming
//            from one scan over the CTA's warps and one over the cluster.  Keys
//            stay in shared memory between the rounds as far as they fit.
//   move     one warp per 16-row group of the new pages gathers its rows and
//            writes the group's contiguous bytes.
// Both are bound by latency and HBM: 4 B of score per (row, head), then 144 B
// read and written per kept row (256 B for FP8).  Nothing is atomic in global
// memory, so the result does not depend on timing.
#include <cooperative_groups.h>

#include "common.cuh"
#include "flat_plan.cuh"
#include "kernels.h"

namespace nvfp4kv {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kKeyCache = 16384;            // keys of a CTA's part kept in shared memory (64 KB)
constexpr int kMaxCluster = 8;
constexpr int kTargetCtasSel = 304;         // two CTAs per SM of a 152-SM GPU

struct SelectArgs {
    const float *scores;
    int64_t score_stride;
    int B, Hkv;
    const int32_t *seq_lens;
    int64_t cap;                // rows a sequence may have: min(table, score_stride)
    int keep, recent, sink;
    int32_t *new_lens, *kept;
    float *new_scores;
    int64_t new_score_stride;
    unsigned *err;
};

// Keys order as the scores do (-0 below +0 would split equal scores: both give
// the key of 0); a NaN gets 0, below -inf.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.0f);   // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(SelectArgs a) {
    extern __shared__ uint32_t s_keys[];            // [kKeyCache]
    __shared__ uint32_t s_hist[256];                // this CTA's counts of a round; read by the cluster
    __shared__ uint32_t s_sum[256];
    __shared__ uint32_t s_warp[kSelWarps][2];       // kept-for-sure and border keys of each warp's part
    __shared__ uint32_t s_cta[2];                   // their sums; read by the cluster
    __shared__ uint32_t s_digit[2];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
    const int seg = (int)blockIdx.y;                // b * Hkv + h
    const int b = seg / a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t len = a.seq_lens[b];
    const int n = clamp_rows(len, a.cap);
    const float *src = a.scores + (int64_t)seg * a.score_stride;
    int32_t *kept = a.kept + (int64_t)seg * a.keep;
    float *dst = a.new_scores + (int64_t)seg * a.new_score_stride;
    const int new_n = min(n, a.keep);
    if (rank == 0 && tid == 0 && seg % a.Hkv == 0) {
        a.new_lens[b] = new_n;
        if (len < 0 || (int64_t)len > a.cap) flag_error(a.err, kErrSeqLen);
    }
    // behind the kept rows: -1 and score 0
    for (int64_t i = new_n + (int64_t)rank * kSelThreads + tid; i < a.new_score_stride; i += (int64_t)C * kSelThreads) {
        dst[i] = 0.f;
        if (i < a.keep) kept[i] = -1;
    }
    if (n <= a.keep) {                              // uniform over the cluster: every row stays
        for (int i = rank * kSelThreads + tid; i < n; i += C * kSelThreads) {
            kept[i] = i;
            dst[i] = src[i];
        }
        return;
    }
    // this CTA's rows [r0, r1), this warp's [w0, w1)
    const int per = (n + C - 1) / C;
    const int r0 = min(n, rank * per), r1 = min(n, r0 + per);
    const int wper = ((r1 - r0 + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int w0 = min(r1, r0 + warp * wper), w1 = min(r1, w0 + wper);
    const int last = n - a.recent;
    auto make_key = [&](int t) { return t < a.sink || t >= last ? 0xffffffffu : score_key(__ldg(src + t)); };
    auto key_of = [&](int t) { return t - r0 < kKeyCache ? s_keys[t - r0] : make_key(t); };

    uint32_t prefix = 0;                            // digits of the border key found so far
    uint32_t need = (uint32_t)a.keep;               // rows still to take among the keys with that prefix
    for (int round = 0; round < 4; round++) {
        const int shift = 24 - 8 * round;
        if (tid < 256) s_hist[tid] = 0;
        __syncthreads();
        for (int tw = w0; tw < w1; tw += 32) {
            const int t = tw + lane;
            uint32_t k = 0;
            bool in = t < w1;
            if (in && round == 0) {
                k = make_key(t);
                if (t - r0 < kKeyCache) s_keys[t - r0] = k;   // read back by this thread only
            } else if (in) {
                k = key_of(t);
                in = (k >> (shift + 8)) == prefix;
            }
            // counts of equal digits are added by one lane (scores share exponents: plain atomics would queue)
            const uint32_t d = in ? (k >> shift) & 255u : 256u;
            const unsigned peers = __match_any_sync(0xffffffffu, d);
            if (in && lane == __ffs(peers) - 1) atomicAdd(&s_hist[d], (uint32_t)__popc(peers));
        }
        cluster.sync();
        if (tid < 256) {
            uint32_t sum = 0;
            for (int r = 0; r < C; r++) sum += cluster.map_shared_rank(s_hist, r)[tid];
            s_sum[tid] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            // the digit whose keys cross `need`, counted from the largest: lane i owns digits 255 - 8i .. 248 - 8i
            uint32_t own = 0;
#pragma unroll
            for (int x = 0; x < 8; x++) own += s_sum[255 - 8 * lane - x];
            uint32_t incl = own;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, x);
                if (lane >= x) incl += y;
            }
            uint32_t above = incl - own;
            if (above < need && need <= incl) {
                for (int x = 0; x < 8; x++) {
                    const uint32_t c = s_sum[255 - 8 * lane - x];
                    if (above + c >= need) {
                        s_digit[0] = 255 - 8 * lane - x;
                        s_digit[1] = need - above;
                        break;
                    }
                    above += c;
                }
            }
        }
        cluster.sync();                             // every CTA has read the counts; the digit is published
        prefix = (prefix << 8) | s_digit[0];
        need = s_digit[1];
    }
    // keys above `prefix` all stay, `need` of those equal to it (in index order)
    uint32_t gt = 0, eq = 0;
    for (int t = w0; t < w1; t += 32) {
        const bool in = t + lane < w1;
        const uint32_t k = in ? key_of(t + lane) : 0u;
        gt += (uint32_t)__popc(__ballot_sync(0xffffffffu, in && k > prefix));
        eq += (uint32_t)__popc(__ballot_sync(0xffffffffu, in && k == prefix));
    }
    if (lane == 0) {
        s_warp[warp][0] = gt;
        s_warp[warp][1] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t x = 0, y = 0;
        for (int w = 0; w < kSelWarps; w++) {
            x += s_warp[w][0];
            y += s_warp[w][1];
        }
        s_cta[0] = x;
        s_cta[1] = y;
    }
    cluster.sync();
    uint32_t at = 0, eq_before = 0;                 // kept rows, border keys before this warp
    for (int r = 0; r < rank; r++) {
        const uint32_t *o = cluster.map_shared_rank(s_cta, r);
        at += o[0];
        eq_before += o[1];
    }
    for (int w = 0; w < warp; w++) {
        at += s_warp[w][0];
        eq_before += s_warp[w][1];
    }
    at += min(eq_before, need);
    cluster.sync();                                 // no CTA leaves while its counts may be read
    for (int t = w0; t < w1; t += 32) {
        const bool in = t + lane < w1;
        const uint32_t k = in ? key_of(t + lane) : 0u;
        const unsigned below = (1u << lane) - 1u;
        const unsigned eqs = __ballot_sync(0xffffffffu, in && k == prefix);
        const bool take = in && (k > prefix || (k == prefix && eq_before + (uint32_t)__popc(eqs & below) < need));
        const unsigned takes = __ballot_sync(0xffffffffu, take);
        if (take) {
            const uint32_t i = at + (uint32_t)__popc(takes & below);
            kept[i] = t + lane;
            dst[i] = __ldg(src + t + lane);
        }
        at += (uint32_t)__popc(takes);
        eq_before += (uint32_t)__popc(eqs);
    }
}

struct MoveArgs {
    uint8_t *pool;
    int64_t num_pages;
    int P, log2P, B, Hkv;
    int64_t slab;
    const int32_t *block_table, *new_block_table;
    int max_pages, new_max_pages, keep;
    const int32_t *kept, *new_lens;
    int dtype;
    unsigned *err;
};

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(MoveArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int groups = (a.keep + 15) / 16;
    const int64_t id = (int64_t)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
    if (id >= (int64_t)a.B * a.Hkv * groups) return;
    const int seg = (int)(id / groups), i0 = (int)(id % groups) * 16;
    const int b = seg / a.Hkv, h = seg % a.Hkv;
    const int rows = min(16, __ldcg(a.new_lens + b) - i0);   // rows of this group that exist
    if (rows <= 0) return;
    const int col = i0 >> a.log2P;
    int64_t page = -1;
    if (col < a.new_max_pages) page = a.new_block_table[(int64_t)b * a.new_max_pages + col];
    if (page < 0 || page >= a.num_pages) {
        if (lane == 0) flag_error(a.err, kErrPage);
        return;
    }
    // lane r < 16 finds the source of row r: its group's address and row (-1: flagged, not moved)
    int64_t src = -1;
    if (lane < rows) {
        const int t = __ldcg(a.kept + (int64_t)seg * a.keep + i0 + lane);
        const int64_t pg = a.block_table[(int64_t)b * a.max_pages + (t >> a.log2P)];
        if (pg < 0 || pg >= a.num_pages) flag_error(a.err, kErrPage);
        else src = (pg << a.log2P) + (t & (a.P - 1));
    }
    const bool fp8 = a.dtype == NVFP4KV_DTYPE_FP8_E4M3;
    const int bytes = fp8 ? 4096 : 2304;
    auto group_of = [&](int64_t slot) {
        const int row = (int)(slot & (a.P - 1));
        return a.pool + ((slot >> a.log2P) * a.Hkv + h) * a.slab + (row >> 4) * bytes;
    };
    uint8_t *dst = a.pool + (page * a.Hkv + h) * a.slab + ((i0 & (a.P - 1)) >> 4) * bytes;
    if (fp8) {   // K 128 bytes a row, then V: 8 chunks of 16 bytes, four rows at a time
#pragma unroll
        for (int x = 0; x < 4; x++) {
            const int r = 4 * x + (lane >> 3), ch = (lane & 7) * 16;
            const int64_t s = __shfl_sync(0xffffffffu, src, r);
            if (s < 0) continue;
            const uint8_t *from = group_of(s) + (s & 15) * 128 + ch;
            const uint4 k = *reinterpret_cast<const uint4 *>(from), v = *reinterpret_cast<const uint4 *>(from + 2048);
            *reinterpret_cast<uint4 *>(dst + r * 128 + ch) = k;
            *reinterpret_cast<uint4 *>(dst + 2048 + r * 128 + ch) = v;
        }
        return;
    }
    // codes: 4 chunks of 16 bytes a row, eight rows at a time, K and V; all loads first
    uint4 k[2], v[2];
    int64_t s[2];
#pragma unroll
    for (int x = 0; x < 2; x++) {
        const int r = 8 * x + (lane >> 2), ch = (lane & 3) * 16;
        s[x] = __shfl_sync(0xffffffffu, src, r);
        if (s[x] < 0) continue;
        const uint8_t *from = group_of(s[x]) + (s[x] & 15) * 64 + ch;
        k[x] = *reinterpret_cast<const uint4 *>(from);
        v[x] = *reinterpret_cast<const uint4 *>(from + 1152);
    }
    // K scales: lane r < 16 its row's 8 bytes.  V scales lie block-major: lane (blk, q) gathers rows 4q .. 4q + 3
    uint2 ks = make_uint2(0, 0);
    if (src >= 0) ks = *reinterpret_cast<const uint2 *>(group_of(src) + 1024 + (src & 15) * 8);
    uint8_t vs[4];
    bool ok[4];
    const int blk = lane >> 2, q = lane & 3;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const int64_t sr = __shfl_sync(0xffffffffu, src, 4 * q + e);
        ok[e] = sr >= 0;
        if (ok[e]) vs[e] = group_of(sr)[2176 + blk * 16 + (sr & 15)];
    }
#pragma unroll
    for (int x = 0; x < 2; x++) {
        const int r = 8 * x + (lane >> 2), ch = (lane & 3) * 16;
        if (s[x] < 0) continue;
        *reinterpret_cast<uint4 *>(dst + r * 64 + ch) = k[x];
        *reinterpret_cast<uint4 *>(dst + 1152 + r * 64 + ch) = v[x];
    }
    if (src >= 0) *reinterpret_cast<uint2 *>(dst + 1024 + lane * 8) = ks;
    uint8_t *vd = dst + 2176 + blk * 16 + 4 * q;
    if (ok[0] && ok[1] && ok[2] && ok[3]) {
        *reinterpret_cast<uchar4 *>(vd) = make_uchar4(vs[0], vs[1], vs[2], vs[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (ok[e]) vd[e] = vs[e];
    }
}

}  // namespace

cudaError_t launch_evict(const nvfp4kv_cache &c, const float *scores, int64_t score_stride, int batch,
                         const int32_t *block_table, int max_pages, const int32_t *seq_lens,
                         const int32_t *new_block_table, int new_max_pages, int keep, int recent, int sink,
                         int32_t *new_lens, int32_t *kept, float *new_scores, int64_t new_score_stride, unsigned *err,
                         cudaStream_t stream) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&select_kernel),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyCache * 4);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    SelectArgs a;
    a.scores = scores;
    a.score_stride = score_stride;
    a.B = batch;
    a.Hkv = c.num_kv_heads;
    a.seq_lens = seq_lens;
    const int64_t table = (int64_t)max_pages * c.page_size;
    a.cap = table < score_stride ? table : score_stride;
    a.keep = keep;
    a.recent = recent;
    a.sink = sink;
    a.new_lens = new_lens;
    a.kept = kept;
    a.new_scores = new_scores;
    a.new_score_stride = new_score_stride;
    a.err = err;
    const int64_t segs = (int64_t)batch * c.num_kv_heads;
    // CTAs a segment: enough to fill the GPU when there are few segments, none with less than 1,024 rows at hand
    int cluster = 1;
    while (cluster < kMaxCluster && segs * cluster < kTargetCtasSel && a.cap >= 2048 * (int64_t)cluster) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster, (unsigned)segs, 1);
    cfg.blockDim = dim3(kSelThreads);
    const int64_t part = ceil_div64(a.cap, cluster);
    cfg.dynamicSmemBytes = (size_t)(part < kKeyCache ? part : kKeyCache) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&a};
    e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(&select_kernel), args);
    if (e != cudaSuccess) return e;

    MoveArgs m;
    m.pool = static_cast<uint8_t *>(c.pool);
    m.num_pages = c.num_pages;
    m.P = c.page_size;
    m.log2P = __builtin_ctz((unsigned)c.page_size);
    m.B = batch;
    m.Hkv = c.num_kv_heads;
    m.slab = (int64_t)(c.dtype == NVFP4KV_DTYPE_NVFP4 ? 144 : 256) * c.page_size;
    m.block_table = block_table;
    m.new_block_table = new_block_table;
    m.max_pages = max_pages;
    m.new_max_pages = new_max_pages;
    m.keep = keep;
    m.kept = kept;
    m.new_lens = new_lens;
    m.dtype = c.dtype;
    m.err = err;
    const int64_t warps = segs * ((keep + 15) / 16);
    void *margs[] = {&m};
    return launch_pdl(reinterpret_cast<const void *>(&move_kernel), (unsigned)ceil_div64(warps, kMoveThreads / 32),
                      kMoveThreads, 0, stream, margs);
}

}  // namespace nvfp4kv
