// gemv.cu -- the forward product of include/moe_ops.h for a few rows (a decode step).
//
//   y[r, n] = act(sum_k x[r, k] W[e, n, k] + bias[n]) + residual[r, n]
//
// With few rows to a weight HBM bounds the call, and the set-up and hand-overs of a tcgen05 tile are
// most of its time (4 x 4096 x 4096: 12.9 us there, 9.6 here, 5.1 at the rate of memory).  Here warps read
// the weights straight into registers, and nothing is set up.  Weights pass once for every eight rows of
// an expert, however many it has; which calls come here is choose_gemv()'s rule (ops.h).
//
// bf16: a warp takes 16 features.  Each lane reads 16-byte pieces of two weight rows and of one row
// of x, in the places that make them operands of mma.m16n8k16 as they are (the order of the
// reduction inside a step is free, so a lane's eight neighbouring values stand for its four
// pairs), eight weight pieces on their way.  On the CUDA cores, four rows took 12.2 us: unpacking
// and multiply-adds, not memory, bounded it.
// fp32: a warp takes two features on the CUDA cores.
// In both, the warps of a block share the reduction where there would be too few of them.  fp32
// sums in a fixed order.
//
// Grouped: a block takes one row as the first of up to eight of its expert's rows, finds the expert by
// looking at all offsets at once, and leaves if the row is not a first one.
#include <cuda_runtime.h>

#include <algorithm>

#include "act.cuh"
#include "common.cuh"
#include "groups.cuh"
#include "ops.h"

namespace moe {
namespace {

constexpr int kThreads = 128;  // fp32
constexpr int kWarps = kThreads / 32;
constexpr int kF = 2;          // features of a warp
constexpr int kRows = 8;
constexpr int kMmaThreads = 256;
constexpr int kMmaWarps = kMmaThreads / 32;
constexpr int kMmaRows = 8;

template <typename T>
struct GemvParams {
  const T* x;
  const T* W;
  const int32_t* offsets;
  const float* bias;
  const T* residual;
  T* y;
  T* preact;
  int64_t R;
  int N, K, E, act;
  int ks;  // warps that share a reduction: a power of two
  Ctrl* ctrl;
};

// The rows of this block: [r0, r0 + rows) of expert e, at most ROWS; false if there is nothing to do.
template <typename T, int ROWS, int THREADS>
__device__ __forceinline__ bool find_rows(const GemvParams<T>& p, int* found, int& r0, int& rows, int& e) {
  if (!p.offsets) {
    e = 0;
    r0 = static_cast<int>(blockIdx.y) * ROWS;
    rows = min(ROWS, static_cast<int>(p.R) - r0);
    return true;
  }
  const int r = static_cast<int>(blockIdx.y);
  if (threadIdx.x == 0) *found = p.E;
  __syncthreads();
  for (int g = threadIdx.x; g < p.E; g += THREADS) {
    int lo, hi;
    if (!group_range(p.offsets, p.R, g, lo, hi)) set_status(p.ctrl, MOE_ERR_DEVICE_BOUNDS);
    if (lo <= r && r < hi) atomicMin(found, g);  // only broken offsets name a row twice
  }
  __syncthreads();
  e = *found;
  if (e == p.E) return false;  // a row of no group
  int lo, hi;
  group_range(p.offsets, p.R, e, lo, hi);
  r0 = r;
  rows = min(ROWS, hi - r);
  return (r - lo) % ROWS == 0;
}

// bias, activation, residual and the stores of one value
template <typename T>
__device__ __forceinline__ void finish(const GemvParams<T>& p, int r, int n, float z) {
  const int64_t at = static_cast<int64_t>(r) * p.N + n;
  if (p.bias) z += __ldg(p.bias + n);
  if (p.preact) p.preact[at] = from_f32<T>(z);
  z = act_f32(z, p.act);
  if (p.residual) z += to_f32(p.residual[at]);
  p.y[at] = from_f32<T>(z);
}

// V consecutive values; those of a weight are read once and not kept in L1, where x is
template <int V>
struct Piece {
  float4 q;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w)
                 : "l"(p));
  }
  __device__ __forceinline__ void keep(const float* p) { q = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void zero() { q = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ float at(int i) const { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; }
};
template <>
struct Piece<1> {  // rows that are not multiples of 16 bytes
  float v;
  __device__ __forceinline__ void load(const float* p) { v = __ldg(p); }
  __device__ __forceinline__ void keep(const float* p) { v = __ldg(p); }
  __device__ __forceinline__ void zero() { v = 0.0f; }
  __device__ __forceinline__ float at(int) const { return v; }
};

// the next kU pieces of both weight rows, from k on
template <int V, int U>
__device__ __forceinline__ void fetch(Piece<V> (*a)[kF], const float* const* w, int k, int step, int K) {
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int f = 0; f < kF; ++f) {
      if (k + u * step < K) a[u][f].load(w[f] + k + u * step);
      else a[u][f].zero();
    }
}

// ROWS: rows computed (a block with fewer repeats its last one)
template <int V, int ROWS>
__device__ __forceinline__ void sum_rows(const float* const* w, const float* const* x, int k, int step, int K,
                                         float (*acc)[kRows]) {
  constexpr int kU = 4;
  Piece<V> a[kU][kF], next[kU][kF];
  fetch<V, kU>(a, w, k, step, K);
  for (; k < K; k += kU * step) {
    fetch<V, kU>(next, w, k + kU * step, step, K);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (k + u * step < K) {
        Piece<V> b[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) b[i].keep(x[i] + k + u * step);
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v)
#pragma unroll
            for (int f = 0; f < kF; ++f) acc[f][i] = fmaf(a[u][f].at(v), b[i].at(v), acc[f][i]);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int f = 0; f < kF; ++f) a[u][f] = next[u][f];
  }
}

template <int V>
__global__ void __launch_bounds__(kThreads) gemv_f32_kernel(const GemvParams<float> p) {
  __shared__ int found;
  __shared__ float part[kWarps][kF * kRows];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int r0, rows, e;
  if (!find_rows<float, kRows, kThreads>(p, &found, r0, rows, e)) return;
  const int fw = warp / p.ks, kw = warp % p.ks;
  const int n0 = (static_cast<int>(blockIdx.x) * (kWarps / p.ks) + fw) * kF;
  // features and rows past the end repeat the last one; their sums are not stored
  const float* w[kF];
  const float* x[kRows];
#pragma unroll
  for (int f = 0; f < kF; ++f) w[f] = p.W + (static_cast<int64_t>(e) * p.N + min(n0 + f, p.N - 1)) * p.K;
#pragma unroll
  for (int i = 0; i < kRows; ++i) x[i] = p.x + static_cast<int64_t>(r0 + min(i, rows - 1)) * p.K;
  float acc[kF][kRows] = {};
  const int step = 32 * V * p.ks, k0 = (kw * 32 + lane) * V;
  if (rows == 1) sum_rows<V, 1>(w, x, k0, step, p.K, acc);
  else if (rows == 2) sum_rows<V, 2>(w, x, k0, step, p.K, acc);
  else if (rows <= 4) sum_rows<V, 4>(w, x, k0, step, p.K, acc);
  else sum_rows<V, kRows>(w, x, k0, step, p.K, acc);
  float mine = 0.0f;  // lane f * kRows + i: the sum of feature f, row i
#pragma unroll
  for (int f = 0; f < kF; ++f)
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float s = acc[f][i];
#pragma unroll
      for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      if (lane == f * kRows + i) mine = s;
    }
  if (p.ks > 1) {
    if (lane < kF * kRows) part[warp][lane] = mine;
    __syncthreads();
    if (kw) return;
    if (lane < kF * kRows)
      for (int q = 1; q < p.ks; ++q) mine += part[warp + q][lane];
  }
  const int n = n0 + lane / kRows, i = lane % kRows;
  if (lane >= kF * kRows || n >= p.N || i >= rows) return;
  finish(p, r0 + i, n, mine);
}

// ------------------------------- bf16 ---------------------------------------------------
__device__ __forceinline__ uint4 ld_once(const __nv_bfloat16* p) {
  uint4 q;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}

__device__ __forceinline__ void mma_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(kMmaThreads, 2) gemv_bf16_kernel(const GemvParams<__nv_bfloat16> p) {
  constexpr int kU = 4;      // chunks on their way
  constexpr int kChunk = 64; // reduction steps: 128 bytes of a row, two pieces a lane
  __shared__ int found;
  __shared__ float4 part[kMmaWarps][32];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  int r0, rows, e;
  if (!find_rows<__nv_bfloat16, kMmaRows, kMmaThreads>(p, &found, r0, rows, e)) return;
  const int fw = warp / p.ks, kw = warp % p.ks;
  const int n0 = (static_cast<int>(blockIdx.x) * (kMmaWarps / p.ks) + fw) * 16;
  // features past the end repeat the last one; their sums are not stored
  const __nv_bfloat16* wl = p.W + (static_cast<int64_t>(e) * p.N + min(n0 + g, p.N - 1)) * p.K + t * 8;
  const __nv_bfloat16* wh = p.W + (static_cast<int64_t>(e) * p.N + min(n0 + g + 8, p.N - 1)) * p.K + t * 8;
  const __nv_bfloat16* x = p.x + static_cast<int64_t>(r0 + g) * p.K + t * 8;
  const bool has = g < rows;
  uint4 lo[kU][2], hi[kU][2];
  auto fetch = [&](int u, int k) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lo[u][h] = hi[u][h] = make_uint4(0, 0, 0, 0);
      if (k + 32 * h + t * 8 < p.K) {
        lo[u][h] = ld_once(wl + k + 32 * h);
        hi[u][h] = ld_once(wh + k + 32 * h);
      }
    }
  };
  const int step = kChunk * p.ks;
  float c[4] = {};
  // The tensor cores cut off what does not fit at each addition: sums of more than kPart turns (of 16
  // additions each) are taken in parts and added in fp32, as in the tiles.
  constexpr int kPart = 64;
#pragma unroll
  for (int u = 0; u < kU; ++u) fetch(u, kw * kChunk + u * step);
  for (int k0 = kw * kChunk, first = k0; k0 < p.K;) {
    const int end = min(p.K, k0 + kPart * kU * step);
    const bool again = k0 != first;
    for (; k0 < end; k0 += kU * step) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int k = k0 + u * step;
        uint4 b[2];  // from L1, except the first time
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          b[h] = make_uint4(0, 0, 0, 0);
          if (has && k + 32 * h + t * 8 < p.K) b[h] = __ldg(reinterpret_cast<const uint4*>(x + k + 32 * h));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_16816(c, lo[u][h].x, hi[u][h].x, lo[u][h].y, hi[u][h].y, b[h].x, b[h].y);
          mma_16816(c, lo[u][h].z, hi[u][h].z, lo[u][h].w, hi[u][h].w, b[h].z, b[h].w);
        }
        fetch(u, k + kU * step);
      }
    }
    if (again) {  // the parts before, each lane's in a place of its own
      const float4 s = part[warp][lane];
      c[0] += s.x;
      c[1] += s.y;
      c[2] += s.z;
      c[3] += s.w;
    }
    if (k0 < p.K) {
      part[warp][lane] = make_float4(c[0], c[1], c[2], c[3]);
      c[0] = c[1] = c[2] = c[3] = 0.0f;
    }
  }
  if (p.ks > 1) {
    part[warp][lane] = make_float4(c[0], c[1], c[2], c[3]);
    __syncthreads();
    if (kw) return;
    for (int w = 1; w < p.ks; ++w) {
      const float4 s = part[warp + w][lane];
      c[0] += s.x;
      c[1] += s.y;
      c[2] += s.z;
      c[3] += s.w;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // features g and g + 8, rows 2 t and 2 t + 1
    const int n = n0 + g + 8 * (i >> 1), r = 2 * t + (i & 1);
    if (n < p.N && r < rows) finish(p, r0 + r, n, c[i]);
  }
}

template <typename T>
GemvParams<T> params(const GemmArgs& a) {
  return GemvParams<T>{static_cast<const T*>(a.rows), static_cast<const T*>(a.other), a.offsets, a.bias,
                       static_cast<const T*>(a.residual), static_cast<T*>(a.out), static_cast<T*>(a.preact),
                       a.R, a.N, a.K, a.E, a.act, 1, a.ctrl};
}

// Grid of blocks of `warps` warps with `features` a warp: as few warps to a reduction (ks, at least
// `span` reduction steps each) as still make `enough` blocks.
dim3 grid_of(const GemmArgs& a, int rows, int warps, int features, int span, int64_t enough, int& ks) {
  const int64_t units = a.offsets ? a.R : (a.R + rows - 1) / rows;  // blocks in y; at most that many have work
  auto blocks = [&](int k) { return (a.N + warps / k * features - 1) / (warps / k * features); };
  for (ks = 1; ks < warps && units * blocks(ks) < enough && a.K >= span * ks * 2;) ks *= 2;
  return dim3(static_cast<unsigned>(blocks(ks)), static_cast<unsigned>(units));
}

template <int V>
cudaError_t launch_f32(const GemmArgs& a, cudaStream_t st) {
  GemvParams<float> p = params<float>(a);
  // three blocks an SM, each lane with 16 pieces on their way, keep memory busy
  const dim3 grid = grid_of(a, kRows, kWarps, kF, 32 * V, static_cast<int64_t>(a.num_sms) * 3, p.ks);
  count_launches(1);
  return launch_pdl(gemv_f32_kernel<V>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace

cudaError_t launch_gemv(const GemmArgs& a, bool bf16, cudaStream_t st) {
  if (!bf16) return a.K % 4 == 0 ? launch_f32<4>(a, st) : launch_f32<1>(a, st);
  GemvParams<__nv_bfloat16> p = params<__nv_bfloat16>(a);
  const dim3 grid = grid_of(a, kMmaRows, kMmaWarps, 16, 128, static_cast<int64_t>(a.num_sms) * 3 / 2, p.ks);
  count_launches(1);
  return launch_pdl(gemv_bf16_kernel, grid, dim3(kMmaThreads), 0, st, p);
}

}  // namespace moe
