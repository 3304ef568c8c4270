// latent.cuh -- sizes of the latent cache format (include/nvfp4kv.h).
#pragma once

namespace nvfp4kv {

constexpr int kLatentDim = 512;            // latent values a token (NVFP4)
constexpr int kRopeDim = 64;               // rotary values a token (BF16)
constexpr int kLatentRow = 416;            // bytes a token: 256 codes, 32 scales, 128 rotary
constexpr int kLatentGroup = 16 * kLatentRow;  // a group of 16 rows: codes [8][16][32] | scales [16][32] | rotary [16][128]
constexpr int kLatentScales = 4096;        // offset of a group's scales
constexpr int kLatentRope = 4608;          // offset of a group's rotary parts

}  // namespace nvfp4kv
