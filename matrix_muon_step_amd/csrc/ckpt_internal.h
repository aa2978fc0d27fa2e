// 8-bit activation checkpoints and the weight gradient that reads them: what
// the host and the kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

// A checkpoint holds blocks of 32 tokens x 32 columns, 1024 bytes each, block
// (R, S) of ceil(tokens / 32) x ceil(cols / 32) at (R * nS + S) * 1024, then
// one exponent byte per block in the same order.  Inside a block, byte
// 16 (32 h + n) + 8 s + i holds token 16 s + 8 h + i of column n: the 16
// bytes of lane 32 h + n are its right operands of two 32x32x16 products
// (s = 0, 1) with the tokens as the summed index, so the gradient product
// reads whole blocks as they lie.  Places past the last token or column hold
// zero.
constexpr int kCkTile = 32;
constexpr int kCkBlockBytes = 1024;
// The smallest exponent keeps every held value a normal bfloat16 number.
constexpr int kCkMinExp = -117;

// One activation of a write or read launch: 32 x 256 of it per work-group.
constexpr int kCkGroupCols = 256;
constexpr int kCkBatch = 32;
struct CkDesc {
  unsigned char* x;
  int64_t stride;        // elements
  unsigned char* codes;
  unsigned char* exps;
  int32_t tokens, cols;
  int32_t blocks;        // blocks of a row of blocks (nS)
  int32_t groups;        // work-groups along the columns
  int32_t f32;           // x is float32 (else bfloat16)
  int32_t pad;
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
  float* part;           // splits > 1: splits x outs x cols partial sums
  int32_t tokens, outs, cols;
  int32_t blocks;        // nS of the checkpoint
  int32_t mt, nt;        // tiles along outs and cols
  int32_t splits;        // parts of the token range
  int32_t per_split;     // 32-token steps of a part
  int32_t g_f32, accumulate;
};
struct GradBatch {
  GradDesc d[kGradBatch];
  int32_t prefix[kGradBatch + 1];   // work-groups of the product
  int32_t sums[kGradBatch + 1];     // work-groups of the joining pass
  int32_t n;
};
// Tile of the product kernel (outs x cols).
constexpr int kGradTile = 256;
hipError_t launch_ckpt_grad(const GradBatch& b, bool aligned, hipStream_t s);
constexpr int kGradSumElems = 2048;  // elements of G per work-group of the joining pass
hipError_t launch_grad_join(const GradBatch& b, hipStream_t s);

}  // namespace muon
