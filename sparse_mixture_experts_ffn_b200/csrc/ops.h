// ops.h -- host-side launch interface between the C ABI of include/moe_ops.h (ops_api.cu)
// and its kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "moe_ops.h"

namespace moe {

// the three products of y = x W^T and its gradients
enum GemmPass { kFwd = 0, kDgrad = 1, kWgrad = 2 };

struct GemmArgs {
  GemmPass pass;
  int64_t R;
  int N, K, E;
  const void* rows;        // fwd: x [R, K]; dgrad, wgrad: dy [R, N]
  const void* other;       // fwd, dgrad: W [E, N, K]; wgrad: x [R, K]
  const int32_t* offsets;  // [E + 1], or null: one group of all R rows
  void* out;               // fwd: y [R, N]; dgrad: dx [R, K]; wgrad: dW [E, N, K]
  // forward epilogue: z = acc + bias, out = act(z) + residual
  const float* bias;       // [N] or null
  const void* residual;    // [R, N] or null; may be out
  void* preact;            // [R, N] or null: receives z
  int act;
  int num_sms;
  Ctrl* ctrl;
};
cudaError_t launch_gemm_bf16(const GemmArgs& a, cudaStream_t st);
cudaError_t launch_gemm_f32(const GemmArgs& a, cudaStream_t st);
// The forward product for a few rows: weights pass once for every eight rows of an expert.
cudaError_t launch_gemv(const GemmArgs& a, bool bf16, cudaStream_t st);
// Measured against the tiles, in us, with the rows spread evenly / all with one expert (the sizes of the
// groups are not known here, only their average):
//                                     few-row kernel   tiles
//   bf16, 288 of 2560 x 4096, 1 row     879 / 102    882 / 27
//                             2 rows    887 / 189    911 / 51
//         288 of 512 x 512,   2 rows     31 / 15      33 / 8
//                             4 rows     35 / 24      33 / 8
//   fp32, 16 of 1024 x 1024,  1 row      12 / 8       90 / 42 (row tiles are mostly padding)
//                             8 rows     39 / 39     111 / 65
//         288 of 1024 x 1024, 8 rows    716 / 694    965 / 287
//         288 of 512 x 512,   8 rows    280 / 279    251 / 83
//         64 of 512 x 512,    16 rows   109 / 108     65 / 51
//   linear layer, bf16, 8 rows of 2048 x 2048 4.1 and 8.5, 16 rows of 11264 x 4096 32 and 24;
//                 fp32, 16 rows of 2048 x 2048 12 and 27
// So the rule is for spread rows.  With all of them at one expert the few-row kernel never takes
// longer than with as many spread, but up to five times as long as the tiles would.
inline bool choose_gemv(const GemmArgs& a, bool bf16) {
  if (a.pass != kFwd) return false;
  if (!a.offsets) return a.R <= (bf16 ? 8 : 16);
  return a.R <= static_cast<int64_t>(a.E) * (bf16 ? 2 : 8);
}

struct SwigluArgs {
  bool bf16;
  int64_t R;
  int I;
  const void* dh;       // backward only
  const void* gate_up;
  const float* row_w;   // or null
  float limit;          // 0: none
  void* out;            // h, or d_gate_up
  float* d_row_w;       // backward only, or null
};
cudaError_t launch_swiglu(const SwigluArgs& a, cudaStream_t st);
cudaError_t launch_swiglu_backward(const SwigluArgs& a, cudaStream_t st);

// dz = dy act'(z) (dz null: not stored; act none: dz = dy is not stored either) and, where
// dbias is not null, its column sums through `partial` (dact_chunks(R) x N floats)
struct DactArgs {
  bool bf16;
  int64_t R;
  int N, act;
  const void* dy;
  const void* z;
  void* dz;
  float* dbias;
  float* partial;
};
int dact_chunks(int64_t R, int N);
cudaError_t launch_dact(const DactArgs& a, cudaStream_t st);

}  // namespace moe
