// accept.cu -- the accepted drafts of each sequence moved together behind its prefix.
//
// A sequence's last d cached tokens are drafts.  Row n - d + accepted[k] becomes row n - d + k,
// for k < num_accepted: 144 bytes (NVFP4) a row and kv head, moved as they are.  A few
// rows a sequence: latency alone.  One warp per (sequence, kv head, part of a row) -- K codes,
// V codes, scales -- loads all of its part's rows (64 at most) before it stores the first, so
// any order and repeated entries are right and nothing is staged in shared memory.  6.8 us for one
// sequence, 8.8 us for 128 with up to 60 drafts and 8 kv heads (cold caches): list, page and
// row are read one after the other.
#include "common.cuh"
#include "kernels.h"

namespace nvfp4kv {

namespace {

constexpr int kWarpsA = 4;      // warps a CTA; a warp takes one part of one kv head

struct AcceptArgs {
    uint8_t *pool;
    int64_t num_pages, slab;
    int P, log2P, Hkv, max_pages, max_accept;
    const int32_t *block_table, *seq_lens, *cu_q, *accepted, *num_accepted;
    int32_t *new_lens;
    unsigned *err;
};

// kFp8: 128-byte rows of codes, two parts; else 64-byte rows and the scales, three.
template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarpsA) accept_kernel(AcceptArgs a) {
    constexpr int kParts = kFp8 ? 2 : 3, kGroup = kFp8 ? 4096 : 2304, kRow = kFp8 ? 128 : 64;
    constexpr int kPieces = kRow / 16, kPer = kMaxDrafts * kPieces / 32;   // 16-byte pieces of a row, and a lane's
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const int job = blockIdx.x * kWarpsA + (threadIdx.x >> 5);
    if (job >= a.Hkv * kParts) return;
    const int head = job / kParts, part = job - head * kParts;
    const bool first = job == 0 && lane == 0;
    const int64_t cap = (int64_t)a.max_pages * a.P;
    const int32_t len = a.seq_lens[b];
    const int n = len < 0 ? 0 : (int64_t)len > cap ? (int)cap : len;
    const int64_t d64 = (int64_t)a.cu_q[b + 1] - a.cu_q[b];
    int count = a.num_accepted[b];
    bool bad_len = len < 0 || (int64_t)len > cap, bad = count < 0 || count > a.max_accept || d64 < 0 || d64 > kMaxDrafts || d64 > n;
    const int d = d64 < 0 || d64 > kMaxDrafts || d64 > n ? 0 : (int)d64, base = n - d;
    count = max(0, min(count, min(a.max_accept, kMaxDrafts)));
    // lane: entries lane and lane + 32; the first that is no draft ends the list
    int from[2];
    int valid = count;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int k = lane + 32 * i;
        from[i] = k < count ? a.accepted[(int64_t)b * a.max_accept + k] : 0;
        const unsigned wrong = __ballot_sync(0xffffffffu, k < count && (from[i] < 0 || from[i] >= d));
        if (wrong) valid = min(valid, 32 * i + __ffs(wrong) - 1);
    }
    if (valid > d) valid = d;                     // (repeated entries may be more than there are rows)
    bad = bad || valid < a.num_accepted[b];
    if (first) {
        a.new_lens[b] = base + valid;
        if (bad_len) flag_error(a.err, kErrSeqLen);
        if (bad) flag_error(a.err, kErrDraft);
    }
    // the group and row of position t; nullptr if its page is out of range
    auto row_of = [&](int t, int &r) -> uint8_t * {
        const int32_t pg = __ldg(a.block_table + (int64_t)b * a.max_pages + (t >> a.log2P));
        r = t & 15;
        if (pg < 0 || (int64_t)pg >= a.num_pages) {
            if (part == 0 && head == 0) flag_error(a.err, kErrPage);
            return nullptr;
        }
        return a.pool + ((int64_t)pg * a.Hkv + head) * a.slab + (int64_t)((t & (a.P - 1)) >> 4) * kGroup;
    };
    if (kFp8 || part < 2) {
        uint4 x[kPer];
        uint8_t *to[kPer];
        const int at = kFp8 ? part * 2048 : part * 1152;
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const int k0 = i * (32 / kPieces), k = k0 + lane / kPieces, piece = lane % kPieces;
            to[i] = nullptr;
            if (k0 >= valid) continue;            // (the same for the whole warp)
            // a lane's entries lie in one of the two registers: k0 / 32 does not depend on the lane
            const int src = __shfl_sync(0xffffffffu, k0 < 32 ? from[0] : from[1], k & 31);
            if (k >= valid || src == k) continue;
            int rs, rd;
            const uint8_t *s = row_of(base + src, rs);
            uint8_t *t = row_of(base + k, rd);
            if (!s || !t) continue;
            x[i] = *reinterpret_cast<const uint4 *>(s + at + rs * kRow + piece * 16);
            to[i] = t + at + rd * kRow + piece * 16;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (to[i]) *reinterpret_cast<uint4 *>(to[i]) = x[i];
    } else {
        uint2 ks[2], vs[2];
        uint8_t *to[2];
        int row[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int k = lane + 32 * i;
            to[i] = nullptr;
            row[i] = 0;
            if (k >= valid || from[i] == k) continue;
            int rs;
            const uint8_t *s = row_of(base + from[i], rs);
            uint8_t *t = row_of(base + k, row[i]);
            if (!s || !t) continue;
            ks[i] = *reinterpret_cast<const uint2 *>(s + 1024 + rs * 8);
            uint32_t lo = 0, hi = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) {         // V scales [block][row]
                lo |= (uint32_t)s[2176 + e * 16 + rs] << (8 * e);
                hi |= (uint32_t)s[2176 + (e + 4) * 16 + rs] << (8 * e);
            }
            vs[i] = make_uint2(lo, hi);
            to[i] = t;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (!to[i]) continue;
            *reinterpret_cast<uint2 *>(to[i] + 1024 + row[i] * 8) = ks[i];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                to[i][2176 + e * 16 + row[i]] = (uint8_t)(vs[i].x >> (8 * e));
                to[i][2176 + (e + 4) * 16 + row[i]] = (uint8_t)(vs[i].y >> (8 * e));
            }
        }
    }
}

}  // namespace

cudaError_t launch_accept(const nvfp4kv_cache &c, const int32_t *block_table, int max_pages, const int32_t *seq_lens,
                          const int32_t *cu_q, int batch, const int32_t *accepted, int max_accept,
                          const int32_t *num_accepted, int32_t *new_lens, unsigned *err, cudaStream_t stream) {
    const bool fp8 = c.dtype == NVFP4KV_DTYPE_FP8_E4M3;
    AcceptArgs a;
    a.pool = static_cast<uint8_t *>(c.pool);
    a.num_pages = c.num_pages;
    a.slab = (int64_t)(fp8 ? 256 : 144) * c.page_size;
    a.P = c.page_size;
    a.log2P = __builtin_ctz((unsigned)c.page_size);
    a.Hkv = c.num_kv_heads;
    a.max_pages = max_pages;
    a.max_accept = max_accept;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.cu_q = cu_q;
    a.accepted = accepted;
    a.num_accepted = num_accepted;
    a.new_lens = new_lens;
    a.err = err;
    void *args[] = {&a};
    const int jobs = c.num_kv_heads * (fp8 ? 2 : 3);
    return launch_pdl(fp8 ? reinterpret_cast<const void *>(&accept_kernel<true>)
                          : reinterpret_cast<const void *>(&accept_kernel<false>),
                      dim3((unsigned)((jobs + kWarpsA - 1) / kWarpsA), (unsigned)batch), 32 * kWarpsA, 0, stream, args);
}

}  // namespace nvfp4kv
