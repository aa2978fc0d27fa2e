// 8-bit activation checkpoints and the weight gradient that reads them: what
// the host and the kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

// A checkpoint holds blocks of 32 tokens x 32 columns, 1024 bytes each, block
// (R, S) of nR x nS = ceil(tokens / 32) x ceil(cols / 32) at (R * nS + S) *
// 1024, then one exponent byte per block, block (R, S) at S * nR + R, so that
// a column block's exponents along the tokens lie together.  Inside a block, byte
// 16 (32 h + n) + 8 s + i holds token 16 s + 8 h + i of column n: the 16
// bytes of lane 32 h + n are its right operands of two 32x32x16 products
// (s = 0, 1) with the tokens as the summed index, so the gradient product
// reads whole blocks as they lie.  Places past the last token or column hold
// zero.
constexpr int kCkTile = 32;
constexpr int kCkBlockBytes = 1024;
// The smallest exponent keeps every held value a normal bfloat16 number.
constexpr int kCkMinExp = -117;
// The exponent of the largest finite float32 inputs.
constexpr int kCkMaxExp = 120;

// One activation of a write or read launch: 32 x 256 of it per work-group.
constexpr int kCkGroupCols = 256;
constexpr int kCkBatch = 32;
struct CkDesc {
  unsigned char* x;
  int64_t stride;        // elements
  unsigned char* codes;
  unsigned char* exps;
  int32_t tokens, cols;
  int32_t blocks;        // nS
  int32_t rblocks;       // nR
  int32_t groups;        // work-groups along the columns
  int32_t f32;           // x is float32 (else bfloat16)
};
struct CkBatch {
  CkDesc d[kCkBatch];
  int64_t prefix[kCkBatch + 1];
  int32_t n;
};
hipError_t launch_ckpt_write(const CkBatch& b, hipStream_t s);
hipError_t launch_ckpt_read(const CkBatch& b, hipStream_t s);

// One matrix of a gradient launch: G (outs x cols) = dY^T X.
constexpr int kGradBatch = 24;
struct GradDesc {
  const unsigned char* dy;
  int64_t dy_stride;     // elements
  const unsigned char* codes;
  const unsigned char* exps;
  unsigned char* G;
  int32_t tokens, outs, cols;
  int32_t blocks;        // nS of the checkpoint
  int32_t mt;            // tiles along outs
  int32_t steps;         // 32-token steps (nR)
  int32_t g_f32, accumulate;
};
// A launch's work is the steps of all tiles of all matrices in a row: tile
// after tile, outs fastest, a tile's steps together.  Either each work-group
// takes one tile (parts == 0), or `parts` work-groups take equal shares, and
// tiles that a share's border cuts are summed from their pieces by a second
// launch.  Piece 2 w of the workspace is the one share w begins with when
// that is inside a tile, piece 2 w + 1 the one it ends with otherwise.
// Matrices without tokens stand behind the others; further work-groups store
// their zeros, a work-group kGradZeros bytes of G (their "tiles").
struct GradBatch {
  GradDesc d[kGradBatch];
  int32_t tiles[kGradBatch + 1];    // exclusive prefix sums of tiles
  int64_t steps[kGradBatch + 1];    // and of their steps
  int64_t share;                    // steps of a work-group (parts > 0)
  float* pieces;
  int32_t parts;
  int32_t n;
  int32_t all;                      // with the matrices without tokens, n ..
};
constexpr int kGradZeros = 65536;
// Square tiles of the product kernels (outs x cols).
enum GradCfg : int32_t { kGrad256 = 0, kGrad128 = 1, kNumGradCfg = 2 };
constexpr int kGradTile[kNumGradCfg] = {256, 128};
hipError_t launch_ckpt_grad(const GradBatch& b, int cfg, bool aligned, hipStream_t s);
hipError_t launch_grad_join(const GradBatch& b, hipStream_t s);  // kGrad256 only

}  // namespace muon
