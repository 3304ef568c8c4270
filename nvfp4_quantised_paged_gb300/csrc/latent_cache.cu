// latent_cache.cu -- BF16 latents -> pages of the latent cache, and back to BF16 rows.
//
// A token of a latent cache is 512 NVFP4 values (32 blocks of 16 with an E4M3
// scale each; quantize.cuh rounds them) and 64 rotary values kept in BF16,
// 416 bytes in the page (the layout is in include/nvfp4kv.h).  Append and
// dequant are bound by HBM: per token 1,152 B of BF16 on one side, 416 B of
// cache on the other.
//
// One warp serves four tokens (two where append rounds under a tensor scale).
// Appending, lane b is block b of each: the 32 lanes read one contiguous kilobyte of a
// token's BF16 row, store its codes in whole 32-byte sectors (four lanes each) and its 32
// scale bytes as one sector.  Expanding, a lane is half a block, so that each store of the
// warp is 512 contiguous bytes (with a block a lane, whose two stores half fill each
// sector, 65,536 tokens took 19.9 us, then 16.6), and the stores are streaming ones
// (14.1): the rows, 75 MB, would push the cache's pages out of L2, and so would the rows
// that append reads (append and expanding one after the other, g 0.75: 46.4 us, with both
// streaming 41.1, now 37.9).  The rotary parts are one 16-byte chunk a lane.  All loads of
// the tokens are issued before the first conversion.
//
// 65,536 tokens: append 14.4 us (7.1 TB/s; 20.2 with a tensor scale, whose roundings
// take their time), expanding 13.7 us (7.5 TB/s, part of it from L2; 17.1).
#include "common.cuh"
#include "kernels.h"
#include "latent.cuh"
#include "quantize.cuh"

namespace nvfp4kv {

namespace {

constexpr int kTokens = 4;                 // tokens per warp, at most
constexpr int kThreads = 256;

struct LatentAppendArgs {
    uint8_t *pool;
    int64_t num_slots;
    int P, log2P;
    const uint4 *latent, *rope;            // BF16 rows viewed as 16-byte vectors
    int64_t latent_stride16, rope_stride16;
    int64_t num_tokens;
    const int64_t *slots;
    float g;
    unsigned *err;
};

// Byte offset of row r's 8 code bytes of block b inside its group.
__device__ __forceinline__ int code_off(int r, int b) { return (b >> 2) * 512 + r * 32 + (b & 3) * 8; }
// Byte offset of row r's scale of block b inside its group.
__device__ __forceinline__ int scale_off(int r, int b) {
    return kLatentScales + r * 32 + ((b >> 1) & 1) * 16 + (b >> 2) * 2 + (b & 1);
}

// Tokens a warp appends: the tensor scale's roundings take registers, and more warps an SM
// make up for fewer tokens each (65,536 tokens: 20.2 us with two, 21.1 with four, 22.3 with
// one; at scale 1 14.9, 14.4 and 15.8).
constexpr int append_tokens(bool unit_scale) { return unit_scale ? kTokens : 2; }

template <bool kUnitScale>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(LatentAppendArgs a) {
    pdl_wait();   // the rows, the slots and the pages may be earlier work's
    pdl_launch_dependents();
    constexpr int NT = append_tokens(kUnitScale);
    const int lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * NT;
    if (t0 >= a.num_tokens) return;
    const int nt = (int)min((int64_t)NT, a.num_tokens - t0);
    uint4 x0[NT], x1[NT], rp = make_uint4(0, 0, 0, 0);
    int64_t slot[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) {
        slot[j] = -1;
        if (j >= nt) continue;
        const uint4 *src = a.latent + (t0 + j) * a.latent_stride16 + lane * 2;
        x0[j] = __ldcs(src);
        x1[j] = __ldcs(src + 1);
        slot[j] = __ldg(a.slots + t0 + j);
    }
    const int rj = lane >> 3, chunk = lane & 7;   // rotary: token and 16-byte chunk of this lane
    if (rj < nt) rp = __ldg(a.rope + (t0 + rj) * a.rope_stride16 + chunk);
    int64_t rslot = -1;
#pragma unroll
    for (int j = 0; j < NT; j++) {
        if (slot[j] >= a.num_slots) {
            if (lane == 0) flag_error(a.err, kErrSlot);
            slot[j] = -1;
        }
        if (j == rj) rslot = slot[j];
        if (slot[j] < 0) continue;
        const int row = (int)(slot[j] & (a.P - 1));
        uint8_t *grp = a.pool + (slot[j] >> a.log2P) * ((int64_t)kLatentRow * a.P) + (row >> 4) * kLatentGroup;
        uint2 codes;
        uint32_t sbyte;
        quantize_block16<kUnitScale>(x0[j], x1[j], a.g, codes, sbyte);
        *reinterpret_cast<uint2 *>(grp + code_off(row & 15, lane)) = codes;
        grp[scale_off(row & 15, lane)] = (uint8_t)sbyte;
    }
    if (rslot >= 0) {
        const int row = (int)(rslot & (a.P - 1));
        uint8_t *grp = a.pool + (rslot >> a.log2P) * ((int64_t)kLatentRow * a.P) + (row >> 4) * kLatentGroup;
        *reinterpret_cast<uint4 *>(grp + kLatentRope + (row & 15) * 128 + ((chunk ^ (row & 7)) << 4)) = rp;
    }
}

struct LatentDequantArgs {
    const uint8_t *pool;
    int64_t num_pages;
    int P, log2P, max_pages, num_reqs;
    const int32_t *block_table, *prefix_lens, *cu;
    int64_t total;
    float g;
    uint4 *latent_ws, *rope_ws;
    unsigned *err;
};

template <bool kUnitScale>
__global__ void __launch_bounds__(kThreads) latent_dequant_kernel(LatentDequantArgs a) {
    pdl_wait();   // the rows, the slots and the pages may be earlier work's
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kTokens;
    if (t0 >= a.total) return;
    // lanes 0..3 find the four tokens' rows in the pool (-1: flagged, not written)
    int64_t src = -1;
    if (lane < kTokens && t0 + lane < a.total) {
        const int64_t row = t0 + lane;
        int lo = 0, hi = a.num_reqs - 1;     // request: the last r with cu[r] <= row
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(a.cu + mid) <= row) lo = mid;
            else hi = mid - 1;
        }
        const int64_t t = row - __ldg(a.cu + lo);
        if (t < 0 || t >= __ldg(a.prefix_lens + lo)) {
            flag_error(a.err, kErrCuPrefix);
        } else if (t >= (int64_t)a.max_pages * a.P) {
            flag_error(a.err, kErrSeqLen);
        } else {
            const int64_t page = __ldg(a.block_table + (int64_t)lo * a.max_pages + (t >> a.log2P));
            if (page < 0 || page >= a.num_pages) flag_error(a.err, kErrPage);
            else src = (page << a.log2P) + (t & (a.P - 1));
        }
    }
    // Lane: half a block (eight values, a 16-byte chunk of the row) at a time, so that a warp's
    // store is contiguous: chunk 32 k + lane of each token.
    uint32_t codes[kTokens][2], sbyte[kTokens][2];
    int64_t slot[kTokens];
#pragma unroll
    for (int j = 0; j < kTokens; j++) {
        slot[j] = __shfl_sync(0xffffffffu, src, j);
        if (slot[j] < 0) continue;
        const int row = (int)(slot[j] & (a.P - 1));
        const uint8_t *grp = a.pool + (slot[j] >> a.log2P) * ((int64_t)kLatentRow * a.P) + (row >> 4) * kLatentGroup;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int b = 16 * k + (lane >> 1);
            codes[j][k] = __ldg(reinterpret_cast<const uint32_t *>(grp + code_off(row & 15, b)) + (lane & 1));
            sbyte[j][k] = __ldg(grp + scale_off(row & 15, b));
        }
    }
    const int rj = lane >> 3, chunk = lane & 7;
    const int64_t rslot = __shfl_sync(0xffffffffu, src, rj);
    if (rslot >= 0) {
        const int row = (int)(rslot & (a.P - 1));
        const uint8_t *grp = a.pool + (rslot >> a.log2P) * ((int64_t)kLatentRow * a.P) + (row >> 4) * kLatentGroup;
        a.rope_ws[(t0 + rj) * 8 + chunk] =
            __ldg(reinterpret_cast<const uint4 *>(grp + kLatentRope + (row & 15) * 128 + ((chunk ^ (row & 7)) << 4)));
    }
#pragma unroll
    for (int j = 0; j < kTokens; j++) {
        if (slot[j] < 0) continue;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            uint32_t o[4];
            nvfp4_half_block_to_bf16<kUnitScale>(codes[j][k], sbyte[j][k], a.g, o);
            __stcs(a.latent_ws + (t0 + j) * (kLatentDim / 8) + 32 * k + lane, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

unsigned grid_of(int64_t tokens, int per_warp) { return (unsigned)ceil_div64(tokens, per_warp * (kThreads / 32)); }

}  // namespace

cudaError_t launch_latent_append(const nvfp4kv_latent_cache &c, const void *latent, int64_t latent_stride,
                                 const void *rope, int64_t rope_stride, int64_t num_tokens,
                                 const int64_t *slot_mapping, unsigned *err, cudaStream_t stream) {
    LatentAppendArgs a;
    a.pool = static_cast<uint8_t *>(c.pool);
    a.num_slots = c.num_pages * (int64_t)c.page_size;
    a.P = c.page_size;
    a.log2P = __builtin_ctz((unsigned)c.page_size);
    a.latent = static_cast<const uint4 *>(latent);
    a.rope = static_cast<const uint4 *>(rope);
    a.latent_stride16 = latent_stride / 8;
    a.rope_stride16 = rope_stride / 8;
    a.num_tokens = num_tokens;
    a.slots = slot_mapping;
    a.g = c.global_scale;
    a.err = err;
    void *args[] = {&a};
    return launch_pdl(c.global_scale == 1.0f ? reinterpret_cast<const void *>(&latent_append_kernel<true>)
                                             : reinterpret_cast<const void *>(&latent_append_kernel<false>),
                      grid_of(num_tokens, append_tokens(c.global_scale == 1.0f)), kThreads, 0, stream, args);
}

cudaError_t launch_latent_dequant(const nvfp4kv_latent_cache &c, const int32_t *block_table, int max_pages,
                                  const int32_t *prefix_lens, const int32_t *cu, int num_reqs, int64_t total,
                                  void *latent_ws, void *rope_ws, unsigned *err, cudaStream_t stream) {
    LatentDequantArgs a;
    a.pool = static_cast<const uint8_t *>(c.pool);
    a.num_pages = c.num_pages;
    a.P = c.page_size;
    a.log2P = __builtin_ctz((unsigned)c.page_size);
    a.max_pages = max_pages;
    a.num_reqs = num_reqs;
    a.block_table = block_table;
    a.prefix_lens = prefix_lens;
    a.cu = cu;
    a.total = total;
    a.g = c.global_scale;
    a.latent_ws = static_cast<uint4 *>(latent_ws);
    a.rope_ws = static_cast<uint4 *>(rope_ws);
    a.err = err;
    void *args[] = {&a};
    return launch_pdl(c.global_scale == 1.0f ? reinterpret_cast<const void *>(&latent_dequant_kernel<true>)
                                             : reinterpret_cast<const void *>(&latent_dequant_kernel<false>),
                      grid_of(total, kTokens), kThreads, 0, stream, args);
}

}  // namespace nvfp4kv
