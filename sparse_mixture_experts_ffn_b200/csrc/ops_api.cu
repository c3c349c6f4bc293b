// ops_api.cu -- the C ABI declared in include/moe_ops.h: validation and launches of the grouped
// products, the linear layer and the gated activation.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <initializer_list>

#include "common.cuh"
#include "ops.h"

namespace moe {
namespace {

// The status word of moe_ops_check_status(), one per device, zero when the library is loaded, and places
// for what its checks took from it: each check has one of its own, as many as may run at a time.
constexpr unsigned kChecks = 1024;
struct OpsWord {
  Ctrl ctrl;
  int taken[kChecks];
};
__device__ OpsWord g_ops_word;

// Reads and clears the word in one step: what another stream's kernel records meanwhile is either
// read now or left for the next check.
__global__ void take_status_kernel(OpsWord* word, unsigned place) {
  word->taken[place] = atomicExch(&word->ctrl.status, 0);
}

OpsWord* ops_word() {
  static std::atomic<void*> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  void* p = cache[dev].load(std::memory_order_acquire);
  if (!p) {
    // the first use on a device may load the module, which a capture on this thread must not forbid
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    const cudaError_t e = cudaGetSymbolAddress(&p, g_ops_word);
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return nullptr;
    cache[dev].store(p, std::memory_order_release);
  }
  return static_cast<OpsWord*>(p);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// a required matrix; an optional one may be null
bool matrix(const void* p) { return p && aligned(p, 16); }
bool optional(const void* p, uintptr_t n) { return aligned(p, n); }

// n bytes from p; null or empty: nothing
struct Span {
  const void* p;
  uint64_t n;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}
// whether an output touches an input or another output
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlap(*o, i)) return true;
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return true;
  }
  return false;
}
uint64_t bytes(int64_t rows, int64_t cols, int32_t dtype) {
  return static_cast<uint64_t>(rows) * static_cast<uint64_t>(cols) * (dtype == MOE_BF16 ? 2 : 4);
}

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int32_t kMaxWidth = 1 << 20;

moe_status check_shape(const moe_gemm_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (s->R < 0 || s->N < 1 || s->K < 1 || s->E < 1) return MOE_ERR_INVALID_ARG;
  if (s->R > kMaxRows || s->N > kMaxWidth || s->K > kMaxWidth || s->E > 1024) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (s->dtype == MOE_BF16 && (s->N % 8 || s->K % 8)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

GemmArgs args_of(const moe_gemm_shape& s, GemmPass pass, const void* rows, const void* other, const int32_t* offsets,
                 void* out) {
  GemmArgs a{};
  a.pass = pass;
  a.R = s.R;
  a.N = s.N;
  a.K = s.K;
  a.E = s.E;
  a.rows = rows;
  a.other = other;
  a.offsets = offsets;
  a.out = out;
  a.num_sms = num_sms_current_device();
  return a;
}

moe_status run_gemm(const moe_gemm_shape& s, GemmArgs a, cudaStream_t st) {
  OpsWord* word = ops_word();
  if (!word) return MOE_ERR_CUDA;
  a.ctrl = &word->ctrl;
  const bool bf16 = s.dtype == MOE_BF16;
  const cudaError_t e = choose_gemv(a, bf16) ? launch_gemv(a, bf16, st) : bf16 ? launch_gemm_bf16(a, st) : launch_gemm_f32(a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status grouped(const moe_gemm_shape* shape, GemmPass pass, const void* rows, const void* other,
                   const int32_t* offsets, void* out, void* stream) {
  const moe_status rc = check_shape(shape);
  if (rc != MOE_OK) return rc;
  if (shape->R == 0 && pass != kWgrad) return MOE_OK;
  // without rows the row operands of a weight gradient are not read and may be null
  if (!offsets || !aligned(offsets, 4) || !matrix(out)) return MOE_ERR_INVALID_ARG;
  if (shape->R > 0 && !(matrix(rows) && matrix(other))) return MOE_ERR_INVALID_ARG;
  const moe_gemm_shape& s = *shape;
  const uint64_t rk = bytes(s.R, s.K, s.dtype), rn = bytes(s.R, s.N, s.dtype);
  const uint64_t w = bytes(static_cast<int64_t>(s.E) * s.N, s.K, s.dtype);
  if (clash({{out, pass == kFwd ? rn : pass == kDgrad ? rk : w}},
            {{rows, pass == kFwd ? rk : rn}, {other, pass == kWgrad ? rk : w}, {offsets, (s.E + 1ull) * 4}}))
    return MOE_ERR_INVALID_ARG;
  return run_gemm(*shape, args_of(*shape, pass, rows, other, offsets, out), static_cast<cudaStream_t>(stream));
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

struct BackwardLayout {
  size_t dz, partial, total;
};
BackwardLayout backward_layout(const moe_gemm_shape& s, int32_t act, bool with_dbias) {
  const size_t es = s.dtype == MOE_BF16 ? 2 : 4;
  BackwardLayout L;
  L.dz = 0;
  L.partial = act == MOE_ACT_NONE ? 0 : align256(static_cast<size_t>(s.R) * s.N * es);
  L.total = L.partial + (with_dbias ? align256(static_cast<size_t>(dact_chunks(s.R, s.N)) * s.N * 4) : 0);
  return L;
}

bool valid_act(int32_t a) { return a >= MOE_ACT_NONE && a <= MOE_ACT_GELU_TANH; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_grouped_gemm(const moe_gemm_shape* shape, const void* x, const void* W,
                                       const int32_t* offsets, void* y, void* stream) {
  return grouped(shape, kFwd, x, W, offsets, y, stream);
}

extern "C" moe_status moe_grouped_gemm_dgrad(const moe_gemm_shape* shape, const void* dy, const void* W,
                                             const int32_t* offsets, void* dx, void* stream) {
  return grouped(shape, kDgrad, dy, W, offsets, dx, stream);
}

extern "C" moe_status moe_grouped_gemm_wgrad(const moe_gemm_shape* shape, const void* dy, const void* x,
                                             const int32_t* offsets, void* dW, void* stream) {
  return grouped(shape, kWgrad, dy, x, offsets, dW, stream);
}

extern "C" moe_status moe_linear(const moe_gemm_shape* shape, const void* x, const void* W, const float* bias,
                                 const void* residual, int32_t activation, void* y, void* preact, void* stream) {
  const moe_status rc = check_shape(shape);
  if (rc != MOE_OK) return rc;
  if (shape->E != 1 || !valid_act(activation)) return MOE_ERR_INVALID_ARG;
  if (shape->R == 0) return MOE_OK;
  if (!matrix(x) || !matrix(W) || !matrix(y) || !optional(bias, 4) || !optional(residual, 16) ||
      !optional(preact, 16))
    return MOE_ERR_INVALID_ARG;
  const uint64_t rn = bytes(shape->R, shape->N, shape->dtype);
  const Span in_x{x, bytes(shape->R, shape->K, shape->dtype)}, in_w{W, bytes(shape->N, shape->K, shape->dtype)};
  const Span in_b{bias, shape->N * 4ull}, in_r{residual, rn};
  if (clash({{y, rn}, {preact, rn}}, {in_x, in_w, in_b})) return MOE_ERR_INVALID_ARG;
  // y may be the residual itself
  if (overlap({preact, rn}, in_r) || (y != residual && overlap({y, rn}, in_r))) return MOE_ERR_INVALID_ARG;
  GemmArgs a = args_of(*shape, kFwd, x, W, nullptr, y);
  a.bias = bias;
  a.residual = residual;
  a.preact = preact;
  a.act = activation;
  return run_gemm(*shape, a, static_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_linear_backward_workspace_bytes(const moe_gemm_shape* shape, int32_t activation,
                                                      int32_t with_dbias) {
  if (check_shape(shape) != MOE_OK || shape->E != 1 || !valid_act(activation)) return 0;
  return backward_layout(*shape, activation, with_dbias != 0).total;
}

extern "C" moe_status moe_linear_backward(const moe_gemm_shape* shape, const void* dy, const void* x, const void* W,
                                          const void* preact, int32_t activation, void* dx, void* dW, float* dbias,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status rc = check_shape(shape);
  if (rc != MOE_OK) return rc;
  const moe_gemm_shape& s = *shape;
  const bool has_act = activation != MOE_ACT_NONE;
  if (s.E != 1 || !valid_act(activation)) return MOE_ERR_INVALID_ARG;
  if (!optional(dx, 16) || !optional(dW, 16) || !optional(dbias, 4)) return MOE_ERR_INVALID_ARG;
  if (s.R > 0 && (!matrix(dy) || (dx && !matrix(W)) || (dW && !matrix(x)) || (has_act && !matrix(preact))))
    return MOE_ERR_INVALID_ARG;
  const BackwardLayout L = backward_layout(s, activation, dbias != nullptr);
  if (L.total) {
    if (!workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  if (dx || dW || dbias) {
    const uint64_t rn = bytes(s.R, s.N, s.dtype), rk = bytes(s.R, s.K, s.dtype), w = bytes(s.N, s.K, s.dtype);
    if (clash({{dx, rk}, {dW, w}, {dbias, s.N * 4ull}, {workspace, L.total}},
              {{dy, rn}, {x, dW ? rk : 0}, {W, dx ? w : 0}, {preact, has_act ? rn : 0}}))
      return MOE_ERR_INVALID_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const void* dz = dy;
  if (dbias || (has_act && (dx || dW) && s.R > 0)) {
    DactArgs d{};
    d.bf16 = s.dtype == MOE_BF16;
    d.R = s.R;
    d.N = s.N;
    d.act = activation;
    d.dy = dy;
    d.z = has_act ? preact : nullptr;
    d.dz = has_act && (dx || dW) ? ws + L.dz : nullptr;
    d.dbias = dbias;
    d.partial = reinterpret_cast<float*>(ws + L.partial);
    if (launch_dact(d, st) != cudaSuccess) return MOE_ERR_CUDA;
    if (d.dz) dz = d.dz;
  }
  if (dx && s.R > 0) {
    const moe_status r = run_gemm(s, args_of(s, kDgrad, dz, W, nullptr, dx), st);
    if (r != MOE_OK) return r;
  }
  if (dW) return run_gemm(s, args_of(s, kWgrad, dz, x, nullptr, dW), st);
  return MOE_OK;
}

static moe_status check_swiglu(int64_t R, int32_t I, int32_t dtype, float limit) {
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || R < 0 || I < 1) return MOE_ERR_INVALID_ARG;
  if (!(limit >= 0.0f) || isinf(limit)) return MOE_ERR_INVALID_ARG;
  if (R > kMaxRows || I > kMaxWidth || (dtype == MOE_BF16 && I % 8)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

extern "C" moe_status moe_swiglu(int64_t R, int32_t I, int32_t dtype, const void* gate_up, const float* row_w,
                                 float limit, void* h, void* stream) {
  const moe_status rc = check_swiglu(R, I, dtype, limit);
  if (rc != MOE_OK || R == 0) return rc;
  if (!matrix(gate_up) || !matrix(h) || !optional(row_w, 4)) return MOE_ERR_INVALID_ARG;
  if (clash({{h, bytes(R, I, dtype)}}, {{gate_up, 2 * bytes(R, I, dtype)}, {row_w, R * 4ull}}))
    return MOE_ERR_INVALID_ARG;
  const SwigluArgs a{dtype == MOE_BF16, R, I, nullptr, gate_up, row_w, limit, h, nullptr};
  return launch_swiglu(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status moe_swiglu_backward(int64_t R, int32_t I, int32_t dtype, const void* dh, const void* gate_up,
                                          const float* row_w, float limit, void* d_gate_up, float* d_row_w,
                                          void* stream) {
  const moe_status rc = check_swiglu(R, I, dtype, limit);
  if (rc != MOE_OK || R == 0) return rc;
  if (!matrix(dh) || !matrix(gate_up) || !matrix(d_gate_up) || !optional(row_w, 4) || !optional(d_row_w, 4))
    return MOE_ERR_INVALID_ARG;
  const uint64_t ri = bytes(R, I, dtype);
  if (clash({{d_gate_up, 2 * ri}, {row_w ? d_row_w : nullptr, R * 4ull}},
            {{dh, ri}, {gate_up, 2 * ri}, {row_w, R * 4ull}}))
    return MOE_ERR_INVALID_ARG;
  const SwigluArgs a{dtype == MOE_BF16, R, I, dh, gate_up, row_w, limit, d_gate_up, row_w ? d_row_w : nullptr};
  return launch_swiglu_backward(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status moe_ops_check_status(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return MOE_ERR_CUDA;
  OpsWord* word = ops_word();
  if (!word) return MOE_ERR_CUDA;
  static std::atomic<unsigned> checks{0};
  const unsigned place = checks.fetch_add(1, std::memory_order_relaxed) % kChecks;
  int status = 0;
  count_launches(1);
  take_status_kernel<<<1, 1, 0, st>>>(word, place);
  if (cudaGetLastError() != cudaSuccess ||
      cudaMemcpyAsync(&status, &word->taken[place], sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return static_cast<moe_status>(status);
}
