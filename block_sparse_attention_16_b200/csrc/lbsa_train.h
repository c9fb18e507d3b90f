// Internal declarations of what a layer has around its attention: rotary
// positions and the per-head norm (rope.cu), the attention's gradients
// (attend_grad.cu, attend_grad_tc.cu).
#pragma once

#include "lbsa_internal.h"

namespace lbsa {

// rotary positions and the per-head norm (rope.cu); strides are in elements: batch, head, row
struct RopeItem {
  const void* x;
  void* y;                 // backward: the gradient of x
  const void* dy;          // backward only
  const void* weight;      // [weight_heads][d] or NULL: no norm
  float* dweight;          // backward only
  int H, rotate, weight_dtype, weight_heads;
  int64_t xs[3], ys[3], ds[3];
};
struct RopePos {
  const float2* table;     // (cos, sin): T x dt/2, then Hg x dh/2, then Wg x dw/2
  int T, Hg, Wg, dt, dh, dw;
  int half;                // pairs (i, i + rd/2) instead of (2i, 2i + 1)
  int tokens;              // T * Hg * Wg; later tokens are not rotated
};
cudaError_t launch_rope(const RopeItem* items, int count, int B, int N, int d, int dtype, const RopePos& pos,
                        const int32_t* perm, float eps, int inverse, int32_t* status, cudaStream_t s);
size_t norm_rope_backward_workspace_bytes(const RopeItem* items, int count, int B, int N, int d, int dtype);
cudaError_t launch_norm_rope_backward(const RopeItem* items, int count, int B, int N, int d, int dtype,
                                      const RopePos& pos, const int32_t* perm, float eps, void* workspace,
                                      int32_t* status, cudaStream_t s);
cudaError_t launch_rope_table(const RopePos& pos, double theta, const double* start, float* table, cudaStream_t s);

// gradients of block-sparse attention (attend_grad.cu)
enum GradTensor { kQ, kK, kV, kOut, kDout, kDq, kDk, kDv, kGradTensors };
struct GradStride {
  int64_t b, h, n;              // elements; the d stride is 1
};
struct AttendGradArgs {
  int B, H, N_valid, d, block, nB;
  const int32_t* counts;
  const int32_t* cols;
  const uint64_t* masks;        // per-token scope, as AttendArgs::masks
  int32_t* status;
  const void *q, *k, *dout;     // bf16: a query tile's own rows are read without a tensor map, k's means taken
  void *dq, *dk, *dv;           // fp32; bf16 gradients leave through tensor maps
  GradStride st[kGradTensors];
  long long wait_limit;
  // the call's tables (attend_grad_workspace)
  int Npad;                     // N_valid rounded up to whole 128-row tiles
  float* neg_lse2;              // [B*H][Npad] -lse in log2 units; -inf: the row keeps nothing
  float* neg_delta;             // [B*H][Npad] -sum of dout * out
  float* k_means;               // bf16: [B*H][Npad / 64][d] mean of each 64 keys, or 0 where they have little in common
  uint32_t* bits;               // [B*H][nB queries][ceil(nB / 32)] kept key blocks
  uint32_t* bits_t;             // [B*H][nB keys][ceil(nB / 32)] query blocks that keep it
  uint64_t* masks_t;            // [B*H][nB keys][nB queries], written where bits are set
};
// sets Npad and, with base, the table pointers; returns the bytes wanted
size_t attend_grad_workspace(AttendGradArgs* a, int dtype, void* base);
cudaError_t launch_attend_grad_prep(const void* out, const void* dout, const float* lse, int dtype,
                                    const AttendGradArgs& a, cudaStream_t s);
// bf16 on the tensor cores (attend_grad_tc.cu); in: q, k, v, dout with boxes of
// 64 columns x 64 rows, out: dq, dk, dv with boxes of 64 x 128
cudaError_t launch_attend_grad_tc(const CUtensorMap* in, const CUtensorMap* out, const AttendGradArgs& a, cudaStream_t s);
cudaError_t launch_attend_grad_f32(const float* q, const float* k, const float* v, const float* dout,
                                   const AttendGradArgs& a, cudaStream_t s);

}  // namespace lbsa
