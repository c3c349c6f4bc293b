// gemm_bf16.cu -- the products of include/moe_ops.h in bf16, on the tensor cores (tcgen05).
//
// One kernel computes all three: a tile is 128 features (the lanes of the accumulator in tensor
// memory) times up to 256 columns,
//   D[m, c] = sum_l A[m, l] B[c, l],   stored as out[c][m]
//   fwd    m = output feature, c = row of the group,  l = input feature    A = W[e],  B = x
//   dgrad  m = input feature,  c = row of the group,  l = output feature   A = W[e]^T, B = dy
//   wgrad  m = input feature,  c = output feature,    l = row of the group A = x^T,   B = dy^T
// Features take the fixed side because they come in multiples of the tile, and rows the other
// because the column count of tcgen05.mma is free in steps of 16: a group of 40 rows costs 48
// columns, not 128.  Transposed operands are not transposed in memory: the matrix descriptors
// of tcgen05 read a tile whose contiguous index is m or c ("MN-major") as well as one whose
// contiguous index is l, so each operand is copied by TMA as it lies.
//
// Blocks are persistent, one an SM: warp 0 copies operands (TMA, 128-byte swizzle) through a ring
// of stages of 64 reduction steps, warp 1 issues the MMAs, warps 2 to 9 move finished tiles from
// tensor memory through shared memory to rows of out, with the forward epilogue on the way; two
// accumulators let the next tile's products run meanwhile.  Tiles are numbered group by group
// (every block computes the prefix of row tiles from the device's offsets) and taken in turn.
//
// SPLIT: where there are too few tiles for the SMs (a decode step), a cluster of 2, 4 or 8 blocks
// shares each tile, each taking a slice of the reduction; the partial tiles are pushed through
// distributed shared memory to the block that owns the column, added there in rank order, and
// finished.  Nothing passes through global memory and no counter needs clearing.
//
// Reading past a group: copies bring whole boxes.  Columns that belong to the next group only
// feed columns of D that are not stored.  Reduction steps past the end are zeros of the copy
// (out-of-bounds fill) for features; for rows (wgrad) the next group's rows are overwritten with
// zeros in shared memory before the last MMAs, so that their values, NaN included, do not count.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "act.cuh"
#include "common.cuh"
#include "groups.cuh"
#include "ops.h"

namespace moe {
namespace {

constexpr int kM = 128;   // features per tile
constexpr int kL = 64;    // reduction steps per stage: 128 bytes of bf16
constexpr int kThreads = 352;
constexpr int kPatchWarp = 10;
constexpr int kABytes = kM * kL * 2;
constexpr int kChunkBytes = kL * 64 * 2;  // an MN-major box: 64 reduction steps x 64 elements
constexpr int kCols = 32;                 // columns per epilogue chunk
// Stages that one accumulator sums.  The tensor cores cut off, not round, what does not fit at every
// addition of 16 steps, so an accumulator's error grows with its length and all one way: up to
// 2^-23 an addition, 2^-13 for these 1024, a 32nd of half a step of bf16.  Longer sums are shared out
// evenly over parts of at most so many stages, added in fp32 (equal terms: in one accumulator,
// 300000 rows were off by 1.6e-3 more than half a step, 10^6 rows by 9.6e-3).  A part costs its tile
// 1 us; parts of 128 stages would cost 4096 x 4096 x 11264 3%.
constexpr int kPart = 256;
constexpr int kMaxSmem = 232448;

// Shared memory of the epilogue's two groups of warps, each: buffers for chunks of 32 columns on
// their way out (wgrad, whose tiles have few reduction steps and wait for their stores, two), and
// with FULL, the epilogue with a residual or a pre-activation, one for pre-activations and two
// for residuals on their way in.
constexpr int kChunk = kCols * kM * 2;
template <int PASS>
constexpr int kOutBufs = PASS == kWgrad ? 2 : 1;
template <int PASS, bool FULL>
constexpr int kGroupBytes = (kOutBufs<PASS> + (FULL ? 3 : 0)) * kChunk;
// The group plan: wgrad reads the offsets where they are, a linear layer (FULL) has one group.
template <int PASS, bool FULL>
constexpr int kPlanGroups = PASS == kWgrad ? 0 : FULL ? 4 : kMaxGroups + 4;

template <int PASS, int BN, bool SPLIT, bool FULL>
struct Cfg {
  static constexpr int kStageBytes = kABytes + BN * kL * 2;
  // or two tiles of pushed partial sums
  static constexpr int kStagingBytes = SPLIT ? 2 * BN * kM * 4 : 2 * kGroupBytes<PASS, FULL>;
  static constexpr int kAuxBytes = 512 + 4 * kPlanGroups<PASS, FULL> * 4;
  static constexpr int kFit = (kMaxSmem - kStagingBytes - 1024 - kAuxBytes) / kStageBytes;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmemBytes = kStages * kStageBytes + kStagingBytes + 1024 + kAuxBytes;
  // Accumulators of one tile.  MMAs that add into the same one wait for each other, which with
  // 16 columns takes longer than the MMA: the four steps of a stage then have one each, added
  // at the end.
  static constexpr int kSums = BN == 16 ? 4 : 1;
  static constexpr int kAccCols = BN * kSums;
  static constexpr int kTmemCols = 2 * kAccCols;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
  static_assert(kStages >= 3 && kSmemBytes <= kMaxSmem, "shared memory budget");
  static_assert(kStageBytes % 1024 == 0, "stages keep the swizzle alignment");
  static_assert(BN % 16 == 0 && BN <= 256, "columns of one MMA");
};

// Division of numbers below 2^31 by a constant of the call: a multiplication and a shift.  With s
// = ceil(log2 d) and mul = ceil(2^(31 + s) / d), which fits 32 bits, n mul / 2^(31 + s) exceeds n / d
// by less than n / 2^31 d < 1 / d, so its integer part is that of n / d.
struct FastDiv {
  uint32_t mul, shift, d;
  FastDiv() = default;
  explicit FastDiv(uint32_t d_) : d(d_) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d_) ++s;
    mul = static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + d_ - 1) / d_);
    shift = 31 + s;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> shift);
  }
};

struct TcParams {
  CUtensorMap tmA, tmB;       // operands
  CUtensorMap tmO, tmR, tmZ;  // out, residual, preact: boxes of 64 features x a chunk's rows
  const int32_t* offsets;
  __nv_bfloat16* out;
  const float* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* preact;
  int64_t R;
  int M, C, L, E;  // features, wgrad's columns per expert, reduction length (fwd, dgrad)
  int bn;          // columns per tile: a multiple of 16 (wgrad: of 64) up to BN
  FastDiv mt;      // feature tiles
  FastDiv ct;      // wgrad: column tiles of an expert
  int ct_band;     // and of a band
  int act;
  Ctrl* ctrl;
};

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// Descriptor of an MN-major operand: boxes of 64 reduction rows of 64 elements (128 B) each,
// swizzled by 128 bytes; 8-row groups 1024 B apart (stride offset), the next 64 elements of the
// other index one box further (leading offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(static_cast<uint32_t>(kChunkBytes) >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

struct Tile {
  int e;
  int m0;        // first feature
  int c0;        // first column: row of the row operand (fwd, dgrad), output feature (wgrad)
  int ncols;     // columns that exist
  int l0;        // wgrad: first row of the group
  int len;       // reduction length
  int64_t orow;  // row of `out` that holds column 0
};

// The group plan in shared memory: the offsets as given, and the row tiles before each group.
struct Plan {
  int* off;    // [E + 1]
  int* start;  // [E + 1] (fwd, dgrad)
  int* per;    // [E] rows of a tile: shared out evenly over the group's tiles, in steps of 16
  int* band;   // [E] row tiles of a band, see band_of()
  // rows [lo, hi) of group e; see group_range()
  template <int PASS>
  __device__ __forceinline__ bool range(const TcParams& p, int e, int& lo, int& hi) const {
    if (PASS == kWgrad) return group_range(p.offsets, p.R, e, lo, hi);
    lo = off[e];
    hi = off[e + 1];
    if (lo < 0 || hi < lo || hi > p.R) {
      lo = hi = 0;
      return false;
    }
    return true;
  }
};

// Order of a group's tiles: the tiles that run at one time (one a pair of SMs, 74) should make a
// block about as high as wide, since what they read is its two edges; what crosses the chip costs
// power, which bounds long runs.  The column tiles are cut into bands of about nine; in a band
// they follow one another, then the features step on.  (4096 x 11264 x 4096 in random data: 365 us
// with the features in the inner place, 16 x 44 tiles; like this 315.)
__host__ __device__ inline int band_of(int tiles) {
  const int bands = (tiles + 4) / 9;
  return bands > 1 ? (tiles + bands - 1) / bands : tiles;
}

// the plan of all groups, by the whole block (ends with a barrier); wgrad: only the check of the offsets
template <int PASS>
__device__ __forceinline__ void make_plan(const TcParams& p, const Plan& plan, int* warp_sums) {
  const int tid = static_cast<int>(threadIdx.x);
  int lo, hi;
  if constexpr (PASS == kWgrad) {  // its tiles do not depend on the rows
    for (int e = tid; e < p.E; e += kThreads)
      if (!plan.template range<PASS>(p, e, lo, hi)) set_status(p.ctrl, MOE_ERR_DEVICE_BOUNDS);
  } else {
    for (int e = tid; e <= p.E; e += kThreads)
      plan.off[e] = p.offsets ? __ldg(p.offsets + e) : (e ? static_cast<int>(p.R) : 0);
    __syncthreads();
    const int per = (p.E + kThreads - 1) / kThreads;
    const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
    int mine = 0;
    for (int e = e0; e < e1; ++e) {
      if (!plan.template range<PASS>(p, e, lo, hi)) set_status(p.ctrl, MOE_ERR_DEVICE_BOUNDS);
      mine += (hi - lo + p.bn - 1) / p.bn;
    }
    const int lane = tid & 31, warp = tid >> 5;
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = incl - mine;
    for (int w = 0; w < warp; ++w) before += warp_sums[w];
    for (int e = e0; e < e1; ++e) {
      plan.template range<PASS>(p, e, lo, hi);
      const int rt = (hi - lo + p.bn - 1) / p.bn;
      plan.start[e] = before;
      plan.per[e] = rt ? ((hi - lo + rt - 1) / rt + 15) & ~15 : 0;
      plan.band[e] = band_of(rt);
      before += rt;
    }
    if (tid == kThreads - 1) plan.start[p.E] = before;
    __syncthreads();
  }
}

// Walks the tiles first, first + step, ... of the schedule; MT: features per tile (a block's 128,
// or a pair's 256).  Tile numbers stay below 2^31: as many tiles would write 2^41 values.
template <int PASS, int MT>
struct Walker {
  const TcParams& p;
  const Plan& plan;
  uint32_t at, step, total;
  int e;
  __device__ __forceinline__ Walker(const TcParams& p_, const Plan& plan_, uint32_t first, uint32_t step_)
      : p(p_), plan(plan_), at(first), step(step_), e(0) {
    total = p.mt.d * (PASS == kWgrad ? p.ct.d * p.E : static_cast<uint32_t>(plan.start[p.E]));
  }
  // tile number `in` of a group of `tiles` column tiles: its column tile, and its feature tile in m
  __device__ __forceinline__ int place(uint32_t in, int tiles, int band, uint32_t& m) const {
    uint32_t b = 0;
    const uint32_t per_band = static_cast<uint32_t>(band) * p.mt.d;
    if (in >= per_band) {
      b = in / per_band;
      in -= b * per_band;
    }
    const int first = static_cast<int>(b) * band;
    const uint32_t n = static_cast<uint32_t>(min(band, tiles - first));
    m = n == 1 ? in : in / n;
    return first + static_cast<int>(in - m * n);
  }
  __device__ __forceinline__ bool next(Tile& r) {
    if (at >= total) return false;
    int lo, hi;
    uint32_t m;
    if (PASS == kWgrad) {
      e = static_cast<int>(p.mt.div(p.ct.div(at)));
      const int c = place(at - static_cast<uint32_t>(e) * (p.mt.d * p.ct.d), static_cast<int>(p.ct.d), p.ct_band, m);
      plan.template range<PASS>(p, e, lo, hi);
      r.c0 = c * p.bn;
      r.ncols = min(p.bn, p.C - r.c0);
      r.l0 = lo;
      r.len = hi - lo;
      r.orow = static_cast<int64_t>(e) * p.C + r.c0;
    } else {
      const int u = static_cast<int>(p.mt.div(at));
      if (u >= plan.start[e + 1]) {  // a later group: the last one that starts by u
        int hi_e = p.E - 1;
        ++e;
        while (e < hi_e) {
          const int mid = (e + hi_e + 1) >> 1;
          if (plan.start[mid] <= u) e = mid;
          else hi_e = mid - 1;
        }
      }
      const int first = plan.start[e];
      const int i = place(at - static_cast<uint32_t>(first) * p.mt.d, plan.start[e + 1] - first, plan.band[e], m);
      plan.template range<PASS>(p, e, lo, hi);
      r.c0 = lo + i * plan.per[e];
      r.ncols = min(plan.per[e], hi - r.c0);
      r.l0 = 0;
      r.len = p.L;
      r.orow = r.c0;
    }
    r.m0 = static_cast<int>(m) * MT;
    r.e = e;
    at += step;
    return true;
  }
};

// store into a block of the cluster, counted in bytes by the mbarrier `bar` of the same block
__device__ __forceinline__ void st_async_f32(uint32_t addr, float v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
               "r"(__float_as_uint(v)), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Waits for the phase of the given parity; CLUSTER: also for what another block of the cluster
// wrote before arriving.  They give up after kWaitLimitNs like mbar_wait(), and look at the timer
// every 256th poll only, so that a wait that is soon over never reads it.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, Ctrl* ctrl, volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 0) {
      if (abort && *abort) return false;
      const uint64_t t = globaltimer_ns();
      if (!t0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        set_status(ctrl, MOE_ERR_DEVICE_TIMEOUT);
        if (abort) *abort = 1;
        return false;
      }
    }
  }
}

// the same by a whole warp, with one answer for all its lanes
template <bool CLUSTER>
__device__ __forceinline__ bool warp_wait_phase(uint64_t* bar, uint32_t parity, Ctrl* ctrl, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_phase<CLUSTER>(bar, parity, ctrl, abort));
}

// rows [from, to) of `boxes` MN-major boxes at `base`: zeros, by one warp
__device__ __forceinline__ void zero_rows(unsigned char* base, int boxes, int from, int to) {
  const int per = (to - from) * 8;
  for (int i = threadIdx.x & 31; i < boxes * per; i += 32) {
    const int box = i / per, at = i - box * per;
    *reinterpret_cast<uint4*>(base + box * kChunkBytes + from * 128 + at * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
}

// 16 lanes x 16 columns of tensor memory as 8-column matrix fragments: registers 4 i .. 4 i + 3 of
// a thread hold, of columns 8 i + 2 (lane % 4) and the next one, row lane / 4 (the first two) and
// row lane / 4 + 8 (the last two).
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// four 8 x 8 matrices of 16-bit values, transposed on the way into shared memory: lanes 8 i .. 8 i
// + 7 give the addresses of the eight 16-byte rows of matrix i
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// the inverse of tmem_ld16_nowait(), and the wait for this thread's stores
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// parts of a sum of nk stages, and the first stage of part i
__device__ __forceinline__ int parts_of(int nk) { return (nk + kPart - 1) / kPart; }
__device__ __forceinline__ int part_begin(int nk, int i, int parts) {
  return static_cast<int>(static_cast<int64_t>(nk) * i / parts);
}

// Adds an accumulator's columns to another's, one lane's row: `width` columns from `first` on, and
// again every `turn`, as the calling warp will read them; SUMS accumulators, BN columns apart.
template <int BN, int SUMS>
__device__ __forceinline__ void add_part(uint32_t to, uint32_t from, int first, int width, int turn, int ncols) {
  for (int c0 = first; c0 < ncols; c0 += turn)
    for (int c = c0; c < min(c0 + width, ncols); c += 16)
#pragma unroll 1
      for (int a = 0; a < SUMS; ++a) {
        uint32_t x[16], y[16];
        float v[16];
        tmem_ld16_nowait(to + c + a * BN, x);
        tmem_ld16_nowait(from + c + a * BN, y);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(x[j]) + __uint_as_float(y[j]);
        tmem_st16(to + c + a * BN, v);
      }
  tmem_wait_st();
}

// columns c .. c + 15 of a tile, one lane's row; BN = 16: the sum of its accumulators
template <int BN>
__device__ __forceinline__ void load_row16(uint32_t trow, int c, int sums, float* v) {
  if constexpr (BN == 16) {
    uint32_t r[4][16];
#pragma unroll
    for (int a = 0; a < 4; ++a) tmem_ld16_nowait(trow + a * BN, r[a]);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      v[j] = __uint_as_float(r[0][j]);
#pragma unroll
      for (int a = 1; a < 4; ++a)
        if (a < sums) v[j] += __uint_as_float(r[a][j]);
    }
  } else {
    tmem_ld16(trow + c, v);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// TMA store of a box {64 features, kCols rows} from shared memory (128-byte swizzle)
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* smem_src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(smem_u32(smem_src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// this thread's stores, except the last N, have read their shared memory
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// this thread's stores are complete
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t* v) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}

// Chunks fetched from tensor memory at a time: a wait is for all fetches.  fwd keeps to one: its
// activation's code is long.
template <int PASS, int BN>
constexpr int kFetched = PASS == kFwd || BN < 4 * kCols ? 1 : 2;
// columns that a group of epilogue warps takes before the other's turn
template <int PASS, int BN>
constexpr int kTaken = kFetched<PASS, BN> * (BN < kCols ? 16 : 32);

// one group of epilogue warps and its shared memory
struct Group {
  int id;              // 0: warps 2 to 5, 1: warps 6 to 9
  unsigned char* out;  // [kOutBufs] chunks
  unsigned char* pre;  // FULL: one chunk
  unsigned char* res;  // FULL: two chunks
  uint64_t* rbar;      // FULL: [2] residual chunk copied
  int buf;
  uint32_t rphase;     // per residual buffer: parity of its next use
  bool leader;         // the thread that issues the group's copies
  __device__ __forceinline__ void sync() const { named_bar_sync(1 + id, 128); }
};

// A finished tile (features m0 .. m0 + 127 in the lanes of tensor memory at `trow`, this warp's
// quarter of them) to rows of `out`, by both groups of four warps, which take chunks of columns in
// turn (one warp for each scheduler of the SM spends most of its time waiting for itself).  sums:
// accumulators that hold the tile; with none the result is zero.  `ready` waits for the
// accumulator; `release` is called by each warp once it has read its part.
//
// The accumulator has features along lanes, `out` has them along rows of memory.  Matrix
// fragments of it are rounded to bf16 and stored through stmatrix, which transposes them, 32
// columns at a time, as two boxes of 64 features (16-byte groups of a 128-byte row permuted by its
// number: the swizzle of the copy, and no bank met twice).  Whole chunks leave by TMA; the
// last chunk of a tile, whose further rows are another group's, by ordinary stores.
// FULL: residual chunks come in by TMA two ahead, ldmatrix brings them into the same fragments, and
// the sum is rounded once; pre-activations leave like the result.
template <int PASS, int BN, bool FULL, typename Ready, typename Release>
__device__ __forceinline__ void store_tile(const TcParams& p, const Tile& tile, int m0, uint32_t trow, int sums,
                                           Group& grp, Ready ready, Release release) {
  constexpr int kHalves = BN < kCols ? 1 : 2;  // no column past the accumulator is read
  constexpr int kStep = 16 * kHalves;
  constexpr int kBlock = kFetched<PASS, BN>;
  constexpr int kTurn = 2 * kBlock * kStep;  // columns of both groups' blocks
  const int et = (threadIdx.x - 64) & 127, lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
  const int group = et & 15, jr = et >> 4;  // ordinary stores: 8 features, every 8th column
  const bool live = m0 + group * 8 < p.M;   // M is a multiple of 8
  const int first = grp.id * kBlock * kStep;
  const bool two = m0 + 64 < p.M;           // boxes of a chunk that exist
  auto load_residual = [&](int c, int b) {  // chunk at column c into buffer b, by the leader
    unsigned char* to = grp.res + b * kChunk;
    mbar_arrive_expect_tx(&grp.rbar[b], (two ? 2u : 1u) * kStep * 128);
    const int row = static_cast<int>(tile.orow) + c;
    tma_load_2d(to, &p.tmR, m0, row, &grp.rbar[b]);
    if (two) tma_load_2d(to + kStep * 128, &p.tmR, m0 + 64, row, &grp.rbar[b]);
  };
  int rb = 0;  // residual buffer of the next chunk
  if (FULL && p.residual && grp.leader) {
    if (first < tile.ncols) load_residual(first, 0);
    if (first + kTurn < tile.ncols) load_residual(first + kTurn, 1);
  }
  float bias[4];  // of features 32 quarter + 8 i + lane / 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + quarter * 32 + 8 * i + (lane >> 2);
    bias[i] = PASS == kFwd && p.bias && m < p.M ? __ldg(p.bias + m) : 0.0f;
  }
  ready();
  if (first >= tile.ncols) {
    if (sums) release();
    return;
  }
  uint32_t r[kBlock][kHalves][16];  // [chunk][16-column half][16-lane half x 8 registers]
  auto fetch = [&](int c0) {
#pragma unroll
    for (int k = 0; k < kBlock; ++k) {
      if (k && c0 + k * kStep >= tile.ncols) break;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int l = 0; l < 2; ++l) {
          if (sums) {
            tmem_ld_frag16(trow + (static_cast<uint32_t>(l * 16) << 16) + c0 + k * kStep + 16 * h, &r[k][h][8 * l]);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) r[k][h][8 * l + q] = 0u;
          }
        }
    }
  };
  fetch(first);
  for (int c0 = first; c0 < tile.ncols; c0 += kTurn) {
    tmem_wait_ld();
    if constexpr (BN == 16) {
      for (int a = 1; a < sums; ++a) {
        uint32_t q[16];
        tmem_ld_frag16(trow + a * BN, q);
        tmem_ld_frag16(trow + (16u << 16) + a * BN, q + 8);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) r[0][0][k] = __float_as_uint(__uint_as_float(r[0][0][k]) + __uint_as_float(q[k]));
      }
    }
    const bool last = c0 + kTurn >= tile.ncols;
    if (sums && last) {  // this group's part of the accumulator has been read
      tc_fence_before();
      __syncwarp();
      release();
    }
#pragma unroll
    for (int k = 0; k < kBlock; ++k) {
      const int c = c0 + k * kStep;
      if (c >= tile.ncols) break;
      unsigned char* st = grp.out + grp.buf * kChunk;
      if (kOutBufs<PASS> == 1) {
        if (grp.leader) bulk_wait_read<0>();  // the last chunk has left
        grp.sync();                           // and nobody reads it
      }
      // where this lane's matrix row of 8-column block b lies in a chunk's buffer
      auto place = [&](int b) {
        const int j = 8 * b + (lane & 7), g = 4 * quarter + (lane >> 3);
        return (g >> 3) * (kStep * 128) + j * 128 + (((g & 7) ^ (j & 7)) << 4);
      };
      float* f = reinterpret_cast<float*>(&r[k][0][0]);
      if (PASS == kFwd && p.bias) {
#pragma unroll
        for (int q = 0; q < 16 * kHalves; ++q) f[q] += bias[2 * ((q >> 3) & 1) + ((q >> 1) & 1)];
      }
      // registers of the features 32 quarter + 8 i + lane / 4 in 8-column block b
      auto pair_at = [&](int b, int i) { return f + 16 * (b >> 1) + 8 * (i >> 1) + 4 * (b & 1) + 2 * (i & 1); };
      auto put = [&](unsigned char* to) {
#pragma unroll
        for (int b = 0; b < 2 * kHalves; ++b) {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = pack_bf16(pair_at(b, i)[0], pair_at(b, i)[1]);
          stmatrix_x4_trans(smem_u32(to + place(b)), v[0], v[1], v[2], v[3]);
        }
      };
      if (FULL && p.preact) put(grp.pre);
      // the choice of activation outside the unrolled values: inside, the code of all five for
      // every value overruns the instruction cache (4096 x 11264 x 4096: 406 us, 359 so)
      if (PASS == kFwd) act_n<16 * kHalves, true>(f, p.act);
      if (FULL && p.residual) {
        wait_phase<false>(&grp.rbar[rb], (grp.rphase >> rb) & 1u, p.ctrl, nullptr);
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 2 * kHalves; ++b) {
          uint32_t v[4];
          ldmatrix_x4_trans(smem_u32(grp.res + rb * kChunk + place(b)), v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            pair_at(b, i)[0] += __uint_as_float(v[i] << 16);
            pair_at(b, i)[1] += __uint_as_float(v[i] & 0xffff0000u);
          }
        }
        grp.rphase ^= 1u << rb;
      }
      put(st);
      if (k == kBlock - 1 && !last) fetch(c0 + kTurn);
      fence_proxy_async_smem();
      if (kOutBufs<PASS> == 2 && grp.leader) bulk_wait_read<0>();  // the other buffer is free
      grp.sync();
      if (FULL && p.residual) {  // everyone has read this chunk's residual
        if (grp.leader && c + 2 * kTurn < tile.ncols) load_residual(c + 2 * kTurn, rb);
        rb ^= 1;
      }
      if (c + kStep <= tile.ncols) {
        if (grp.leader) {
          const int row = static_cast<int>(tile.orow) + c;
          tma_store_2d(&p.tmO, st, m0, row);
          if (two) tma_store_2d(&p.tmO, st + kStep * 128, m0 + 64, row);
          if (FULL && p.preact) {
            tma_store_2d(&p.tmZ, grp.pre, m0, row);
            if (two) tma_store_2d(&p.tmZ, grp.pre + kStep * 128, m0 + 64, row);
          }
          bulk_commit();
        }
      } else {
#pragma unroll
        for (int i = 0; i < kStep / 8; ++i) {
          const int j = jr + 8 * i;
          if (live && c + j < tile.ncols) {
            const int from = (group >> 3) * (kStep * 128) + j * 128 + (((group & 7) ^ (j & 7)) << 4);
            const int64_t at = (tile.orow + c + j) * p.M + m0 + group * 8;
            *reinterpret_cast<uint4*>(p.out + at) = *reinterpret_cast<const uint4*>(st + from);
            if (FULL && p.preact) *reinterpret_cast<uint4*>(p.preact + at) = *reinterpret_cast<const uint4*>(grp.pre + from);
          }
        }
      }
      if (++grp.buf == kOutBufs<PASS>) grp.buf = 0;
    }
  }
}

// whether the phase is over, without waiting
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// What the copying thread has issued, so that it can let its copies land before the block ends: also
// when it has issued them all and another thread's wait failed.
struct InFlight {
  uint32_t used = 0, partial = 0;    // per stage: used at all; its last use was a partial one
  uint32_t whole_odd = 0, part_odd = 0;  // per stage: uses of either kind so far, modulo 2
  __device__ __forceinline__ void issue(int stage, bool part) {
    const uint32_t bit = 1u << stage;
    used |= bit;
    if (part) {
      partial |= bit;
      part_odd ^= bit;
    } else {
      partial &= ~bit;
      whole_odd ^= bit;
    }
  }
  // full null: whole stages land on another block's barriers
  template <int STAGES>
  __device__ __forceinline__ void land(uint64_t* full, uint64_t* qfull, Ctrl* ctrl) const {
    for (int s = 0; s < STAGES; ++s) {
      if (!((used >> s) & 1u)) continue;
      if ((partial >> s) & 1u) wait_phase<false>(&qfull[s], ((part_odd >> s) & 1u) ^ 1u, ctrl, nullptr);
      else if (full) wait_phase<false>(&full[s], ((whole_odd >> s) & 1u) ^ 1u, ctrl, nullptr);
    }
  }
};

// What the MMA thread needs of the ring of stages: descriptors of stage 0, and where it is.
template <int STAGES, int STAGE_BYTES>
struct Ring {
  uint64_t* full;
  uint64_t* empty;
  uint64_t a0, b0;
  int stage;
  uint32_t phases;   // per stage: parity of its next whole use
  uint32_t patched;  // per stage: parity of its next partial use (wgrad)
  __device__ __forceinline__ uint64_t offset() const { return static_cast<uint64_t>(stage) * (STAGE_BYTES >> 4); }
  __device__ __forceinline__ uint32_t parity() const { return (phases >> stage) & 1u; }
  __device__ __forceinline__ void advance() { stage = stage + 1 == STAGES ? 0 : stage + 1; }
};

template <int PASS, bool PAIR>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, int k, uint32_t idesc, uint32_t accumulate) {
  // 16 reduction steps: 32 bytes of a K-major tile, 16 rows of 128 bytes of an MN-major one
  constexpr uint64_t kA = (PASS == kFwd ? 32 : 2048) >> 4, kB = (PASS == kWgrad ? 2048 : 32) >> 4;
  if (PAIR) mma_bf16_pair(d, a + k * kA, b + k * kB, idesc, accumulate);
  else mma_bf16(d, a + k * kA, b + k * kB, idesc, accumulate);
}
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (PAIR) mma_commit_pair(bar);
  else mma_commit(bar);
}

// The MMAs of n whole stages, by one thread; the last has `steps` groups of 16 reduction steps.
// The tensor cores hold few MMAs ahead, so what this thread does between two of them is time they
// may wait: descriptors advance by additions to their address field, four MMAs are unrolled, and
// the next stage's barrier is looked at between the second and the third, while the first ones
// run.  (Descriptors built for every MMA: 217 cycles an MMA of 256 x 256 x 16; like this 161.)
// `pfull` not null: the last stage is a wgrad group's partial one, ready when its barrier there is.
// SUM_COLS: the four steps of a stage add into accumulators of their own, so many columns apart (0:
// all into one).
template <int PASS, bool PAIR, int SUM_COLS, int STAGES, int STAGE_BYTES>
__device__ __forceinline__ bool mma_stages(Ring<STAGES, STAGE_BYTES>& ring, int n, int steps, uint32_t d, uint32_t idesc,
                                           uint64_t* pfull, Ctrl* ctrl, volatile int* abort) {
  bool ready = false;
  for (int i = 0; i < n; ++i) {
    if (PASS == kWgrad && pfull && i + 1 == n) {
      if (!wait_phase<PAIR>(&pfull[ring.stage], (ring.patched >> ring.stage) & 1u, ctrl, abort)) return false;
      ring.patched ^= 1u << ring.stage;
    } else {
      if (!ready && !wait_phase<false>(&ring.full[ring.stage], ring.parity(), ctrl, abort)) return false;
      ring.phases ^= 1u << ring.stage;
    }
    ready = false;
    tc_fence_after();
    const uint64_t a = ring.a0 + ring.offset(), b = ring.b0 + ring.offset();
    uint64_t* done = &ring.empty[ring.stage];
    ring.advance();
    if (i + 1 < n || steps == kL / 16) {
      const uint32_t more = SUM_COLS ? (i ? 1u : 0u) : 1u;
      mma_step<PASS, PAIR>(d, a, b, 0, idesc, i ? 1u : 0u);
      mma_step<PASS, PAIR>(d + SUM_COLS, a, b, 1, idesc, more);
      // (a partial stage's bit says nothing: its barrier is another one)
      ready = i + 1 < n && mbar_test(&ring.full[ring.stage], ring.parity());
      mma_step<PASS, PAIR>(d + 2 * SUM_COLS, a, b, 2, idesc, more);
      mma_step<PASS, PAIR>(d + 3 * SUM_COLS, a, b, 3, idesc, more);
    } else {
      for (int k = 0; k < steps; ++k)
        mma_step<PASS, PAIR>(d + k * SUM_COLS, a, b, k, idesc, i || (k && !SUM_COLS) ? 1u : 0u);
    }
    commit<PAIR>(done);
  }
  return true;
}

template <int PASS, int BN, bool SPLIT, bool FULL>
__global__ void __launch_bounds__(kThreads, 1) gemm_tc_kernel(const __grid_constant__ TcParams p) {
  using C = Cfg<PASS, BN, SPLIT, FULL>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char* staging = smem + C::kStages * C::kStageBytes;
  unsigned char* aux = smem + C::kStages * C::kStageBytes + C::kStagingBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(aux);  // [kStages]
  uint64_t* empty = full + 8;                         // [kStages]
  uint64_t* qfull = empty + 8;                        // [kStages] wgrad: a partial stage copied
  uint64_t* pfull = qfull + 8;                        // [kStages] wgrad: a partial stage patched
  uint64_t* tfull = pfull + 8;                        // [2] accumulator finished
  uint64_t* tempty = tfull + 2;                       // [2] accumulator read
  uint64_t* rfull = tempty + 2;                       // [2] SPLIT: partial sums of all blocks here
  uint64_t* rempty = rfull + 2;                       // [2] SPLIT: every owner has added them
  uint64_t* rbar = rempty + 2;                        // [2 groups][2] FULL: residual chunk copied
  uint64_t* drain = rbar + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* warp_sums = reinterpret_cast<int*>(tmem_slot + 4);
  Plan plan;
  plan.off = reinterpret_cast<int*>(aux + 512);
  constexpr int kPlan = kPlanGroups<PASS, FULL>;
  plan.start = plan.off + kPlan;
  plan.per = plan.start + kPlan;
  plan.band = plan.per + kPlan;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cs = SPLIT ? cluster_size() : 1, rank = SPLIT ? cluster_ctarank() : 0;
  const int cs_log = SPLIT ? 31 - __clz(cs) : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&qfull[s], 1);
      mbar_init(&pfull[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], SPLIT ? 4 : 8);
      mbar_init(&rfull[a], 1);  // and the bytes pushed
      mbar_init(&rempty[a], 4 * cs);
    }
    for (int b = 0; b < 4; ++b) mbar_init(&rbar[b], 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  if (SPLIT) cluster_sync();  // barriers initialised everywhere before any remote arrival
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  make_plan<PASS>(p, plan, warp_sums);
  const uint32_t first = blockIdx.x / cs, step = gridDim.x / cs;
  // this block's slice of a reduction of `len` steps, in stages
  auto slice = [&](int len, int& kb0) {
    const int kb = (len + kL - 1) / kL;
    if (!SPLIT) {
      kb0 = 0;
      return kb;
    }
    kb0 = static_cast<int>(static_cast<int64_t>(kb) * rank / cs);
    return static_cast<int>(static_cast<int64_t>(kb) * (rank + 1) / cs) - kb0;
  };

  if (warp == 0) {
    // ------------------------------- copies --------------------------------------------
    if (lane == 0) {
      const uint32_t bytes = kABytes + static_cast<uint32_t>(p.bn) * kL * 2;
      int stage = 0;
      uint32_t phase = 0;
      InFlight fly;
      bool ok = true;
      Walker<PASS, kM> walk(p, plan, first, step);
      Tile tile;
      while (ok && walk.next(tile)) {
        int kb0;
        const int nk = slice(tile.len, kb0);
        for (int kb = kb0; kb < kb0 + nk; ++kb) {
          if (!wait_phase<false>(&empty[stage], phase ^ 1u, p.ctrl, abort_flag)) { ok = false; break; }
          unsigned char* a = smem + stage * C::kStageBytes;
          unsigned char* b = a + kABytes;
          const bool partial = PASS == kWgrad && tile.len - kb * kL < kL;
          uint64_t* landed = partial ? &qfull[stage] : &full[stage];
          mbar_arrive_expect_tx(landed, bytes);
          if (PASS == kFwd) {
            tma_load_3d(a, &p.tmA, kb * kL, tile.m0, tile.e, landed);
            tma_load_2d(b, &p.tmB, kb * kL, tile.c0, landed);
          } else if (PASS == kDgrad) {
            tma_load_3d(a, &p.tmA, tile.m0, kb * kL, tile.e, landed);
            tma_load_3d(a + kChunkBytes, &p.tmA, tile.m0 + 64, kb * kL, tile.e, landed);
            tma_load_2d(b, &p.tmB, kb * kL, tile.c0, landed);
          } else {
            const int l = tile.l0 + kb * kL;
            tma_load_2d(a, &p.tmA, tile.m0, l, landed);
            tma_load_2d(a + kChunkBytes, &p.tmA, tile.m0 + 64, l, landed);
            for (int c = 0; c < p.bn; c += 64)
              tma_load_2d(b + (c / 64) * kChunkBytes, &p.tmB, tile.c0 + c, l, landed);
          }
          fly.issue(stage, partial);
          if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        }
      }
      fly.land<C::kStages>(full, qfull, p.ctrl);
    }
  } else if (warp == 1) {
    // ------------------------------- MMAs ----------------------------------------------
    if (lane == 0) {
      // D fp32, A and B bf16; bits 15 / 16: A / B is MN-major
      const uint32_t major = (PASS == kFwd ? 0u : 1u << 15) | (PASS == kWgrad ? 1u << 16 : 0u);
      const uint32_t sa = smem_u32(smem), sb = sa + kABytes;  // of stage 0
      Ring<C::kStages, C::kStageBytes> ring{full, empty, PASS == kFwd ? sw128_kmajor_desc(sa) : sw128_mnmajor_desc(sa),
                                            PASS == kWgrad ? sw128_mnmajor_desc(sb) : sw128_kmajor_desc(sb), 0, 0u, 0u};
      int acc = 0;        // accumulator of the tile's first part; further parts take the other one
      uint32_t uses = 0;  // of each accumulator, modulo 2
      bool ok = true;
      Walker<PASS, kM> walk(p, plan, first, step);
      Tile tile;
      while (ok && walk.next(tile)) {
        int kb0;
        const int nk = slice(tile.len, kb0);
        if (nk == 0) continue;  // the epilogue knows: nothing to add
        const uint32_t idesc = idesc_bf16_f32(kM, (tile.ncols + 15) & ~15) | major;
        const int left = min(kL, tile.len - (kb0 + nk - 1) * kL);
        const int parts = parts_of(nk);
        for (int i = 0; i < parts; ++i) {
          const bool last = i + 1 == parts;
          const int a = i ? acc ^ 1 : acc;
          const int n = parts == 1 ? nk : part_begin(nk, i + 1, parts) - part_begin(nk, i, parts);
          ok = wait_phase<false>(&tempty[a], ((uses >> a) & 1u) ^ 1u, p.ctrl, abort_flag);
          if (!ok) break;
          tc_fence_after();
          ok = mma_stages<PASS, false, C::kSums == 1 ? 0 : BN>(ring, n, last ? (left + 15) / 16 : kL / 16,
                                                               tmem_base + a * C::kAccCols, idesc,
                                                               last && left < kL ? pfull : nullptr, p.ctrl, abort_flag);
          if (!ok) break;
          mma_commit(&tfull[a]);
          uses ^= 1u << a;
        }
        acc ^= 1;
      }
      mma_commit(drain);  // every MMA done before the accumulators are freed
      wait_phase<false>(drain, 0, p.ctrl, nullptr);
    }
  } else if (warp == kPatchWarp) {
    if (PASS == kWgrad) {
      // ----------------------------- partial stages ------------------------------------
      int stage = 0;        // of the tile's first reduction steps
      uint32_t phases = 0;  // per stage: parity of its next partial use
      Walker<PASS, kM> walk(p, plan, first, step);
      Tile tile;
      while (walk.next(tile)) {
        int kb0;
        const int nk = slice(tile.len, kb0);
        const int left = tile.len - (kb0 + nk - 1) * kL;
        if (nk > 0 && left < kL) {
          const int at = (stage + nk - 1) % C::kStages;
          if (!warp_wait_phase<false>(&qfull[at], (phases >> at) & 1u, p.ctrl, abort_flag)) break;
          phases ^= 1u << at;
          zero_rows(smem + at * C::kStageBytes, 2 + (tile.ncols + 63) / 64, left, (left + 15) / 16 * 16);
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[at]);
        }
        stage = (stage + nk) % C::kStages;
      }
    }
  } else if (!SPLIT || warp < 6) {
    // ------------------------------- epilogue ------------------------------------------
    // After a failed wait (status set) it goes on without waiting, so that the warps meet at
    // every barrier.
    Group grp{(warp - 2) >> 2, nullptr, nullptr, nullptr, nullptr, 0, 0u, threadIdx.x % 128 == 64};
    grp.out = staging + grp.id * kGroupBytes<PASS, FULL>;
    grp.pre = grp.out + kOutBufs<PASS> * kChunk;
    grp.res = grp.pre + kChunk;
    grp.rbar = rbar + 2 * grp.id;
    const int quarter = warp & 3;            // tensor-memory lanes this warp may read
    const int r = quarter * 32 + lane;       // feature of the tile
    int acc = 0, buf = 0;
    uint32_t uses = 0, buf_phase = 0;
    bool failed = false;
    Walker<PASS, kM> walk(p, plan, first, step);
    Tile tile;
    while (walk.next(tile)) {
      int kb0;
      const int nk = slice(tile.len, kb0);
      const uint32_t trow0 = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
      const uint32_t trow = trow0 + acc * C::kAccCols;
      auto finished = [&](int a) {  // waits for the products in accumulator a
        if (!failed && !wait_phase<false>(&tfull[a], (uses >> a) & 1u, p.ctrl, abort_flag)) failed = true;
        uses ^= 1u << a;
        __syncwarp();
        tc_fence_after();
      };
      auto ready = [&] {
        if (nk == 0) return;
        finished(acc);
        for (int i = 1; i < parts_of(nk); ++i) {
          finished(acc ^ 1);
          constexpr int kWidth = SPLIT ? BN : kTaken<PASS, BN>;
          add_part<BN, C::kSums>(trow, trow0 + (acc ^ 1) * C::kAccCols, SPLIT ? 0 : grp.id * kWidth, kWidth,
                                 SPLIT ? BN : 2 * kWidth, tile.ncols);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc ^ 1]);
        }
      };
      // accumulators written: one for each step of the first stage
      const int sums = nk == 0 ? 0 : C::kSums == 1 || nk > 1 ? C::kSums : (min(kL, tile.len - kb0 * kL) + 15) / 16;
      if constexpr (SPLIT) {
        ready();
        // ---- push this block's partial sums to the columns' owners: column c to block c % cs,
        // which counts the bytes as they arrive
        const int own = (tile.ncols - static_cast<int>(rank) + static_cast<int>(cs) - 1) >> cs_log;
        if (threadIdx.x == 64) mbar_arrive_expect_tx(&rfull[buf], static_cast<uint32_t>(own) * cs * kM * 4);
        if (!failed && !wait_phase<true>(&rempty[buf], buf_phase ^ 1u, p.ctrl, abort_flag)) failed = true;
        __syncwarp();
        float* recv = reinterpret_cast<float*>(staging) + buf * BN * kM;  // [owned column][rank][feature]
        const uint32_t to = smem_u32(recv + rank * kM + r), bar = smem_u32(&rfull[buf]);
        for (int c = 0; c < tile.ncols; c += 16) {
          float v[16];
          if (sums) {
            load_row16<BN>(trow, c, sums, v);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.0f;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (c + j < tile.ncols) {
              const uint32_t col = c + j, q = col & (cs - 1);
              st_async_f32(mapa_shared(to + (((col >> cs_log) << cs_log) * kM) * 4, q), v[j], mapa_shared(bar, q));
            }
          }
        }
        if (sums) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        }
        // ---- add the shares of the columns owned here, in rank order
        constexpr int kOwn = BN / 2;  // two blocks at least
        const int m = tile.m0 + r;
        const bool live = m < p.M;
        const int64_t at0 = (tile.orow + rank) * p.M + m, at_step = static_cast<int64_t>(cs) * p.M;
        const float b = PASS == kFwd && p.bias && live ? __ldg(p.bias + m) : 0.0f;
        __nv_bfloat16 res[kOwn];
        if (PASS == kFwd && p.residual && live) {
#pragma unroll
          for (int i = 0; i < kOwn; ++i)
            if (i < own) res[i] = p.residual[at0 + i * at_step];
        }
        // (also after a failed wait: the blocks push all the same, and none may end before it has landed)
        if (!wait_phase<true>(&rfull[buf], buf_phase, p.ctrl, nullptr)) failed = true;
        __syncwarp();
        float z[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          if (i >= own) break;
          z[i] = 0.0f;
          for (uint32_t q = 0; q < cs; ++q) z[i] += recv[((static_cast<uint32_t>(i) << cs_log) + q) * kM + r];
        }
        __syncwarp();  // the shares have been read (and nothing stored yet that the release would wait for)
        if (lane < static_cast<int>(cs)) mbar_arrive_remote(mapa_shared(smem_u32(&rempty[buf]), lane));
        if (live) {
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            if (i >= own) break;
            const int64_t at = at0 + i * at_step;
            if (PASS == kFwd) {
              z[i] += b;
              if (p.preact) p.preact[at] = __float2bfloat16_rn(z[i]);
              act_n<1, true>(&z[i], p.act);
              if (p.residual) z[i] += __bfloat162float(res[i]);
            }
            p.out[at] = __float2bfloat16_rn(z[i]);
          }
        }
        if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
      } else {
        store_tile<PASS, BN, FULL>(p, tile, tile.m0, trow, sums, grp, ready, [&] {
          if (lane == 0) mbar_arrive(&tempty[acc]);
        });
      }
      if (nk) acc ^= 1;
    }
    bulk_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (SPLIT) cluster_sync();  // no block leaves while another may still write to it
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, C::kTmemCols);
}

// ------------------------------- pairs of SMs -------------------------------------------
// The same tiles twice as high: a cluster of two blocks computes 256 features x up to 256
// columns with tcgen05.mma cta_group::2.  Each block copies its own 128 features and half of
// the columns, so that a stage of 64 reduction steps costs it 32 KB instead of 48 for the same
// products: large tiles are bound by what L2 delivers, not by the tensor cores.  The even
// block issues the MMAs; each block's tensor memory receives its own features.
//
// The copies of both blocks complete on the even block's barrier.  wgrad: those of a group's last,
// partial stage complete at home, where the patch warp zeroes the block's part of the rows past the
// group and tells the even block (passing every stage on that way took longer than its MMAs).
template <int PASS, bool FULL>
struct PairCfg {
  static constexpr int BN = 256;
  static constexpr int kStageBytes = kABytes + BN / 2 * kL * 2;
  static constexpr int kStagingBytes = 2 * kGroupBytes<PASS, FULL>;
  static constexpr int kAuxBytes = 512 + 4 * kPlanGroups<PASS, FULL> * 4;
  static constexpr int kStages = (kMaxSmem - kStagingBytes - 1024 - kAuxBytes) / kStageBytes;
  static constexpr int kSmemBytes = kStages * kStageBytes + kStagingBytes + 1024 + kAuxBytes;
  static_assert(kStages >= 4 && kStages <= 8, "stages");
};

__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, int32_t c0, int32_t c1,
                                                 int32_t c2, uint32_t bar_cluster_addr) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cluster_addr)
      : "memory");
}

// columns that a tile's MMAs compute: half of them (a multiple of 16) from each block
__device__ __forceinline__ int pair_columns(const Tile& t) { return (t.ncols + 31) & ~31; }

template <int PASS, bool FULL>
__global__ void __launch_bounds__(kThreads, 1) gemm_pair_kernel(const __grid_constant__ TcParams p) {
  using C = PairCfg<PASS, FULL>;
  constexpr int MT = 2 * kM;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char* staging = smem + C::kStages * C::kStageBytes;
  unsigned char* aux = smem + C::kStages * C::kStageBytes + C::kStagingBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(aux);  // [kStages] even block: both blocks' copies
  uint64_t* empty = full + 8;                         // [kStages]
  uint64_t* qfull = empty + 8;                        // [kStages] wgrad: own copies of a partial stage
  uint64_t* pfull = qfull + 8;                        // [kStages] wgrad, even block: patched by both
  uint64_t* tfull = pfull + 8;                        // [2]
  uint64_t* tempty = tfull + 2;                       // [2] even block
  uint64_t* rbar = tempty + 2;                        // [2 groups][2] FULL: residual chunk copied
  uint64_t* drain = rbar + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* warp_sums = reinterpret_cast<int*>(tmem_slot + 4);
  Plan plan;
  plan.off = reinterpret_cast<int*>(aux + 512);
  constexpr int kPlan = kPlanGroups<PASS, FULL>;
  plan.start = plan.off + kPlan;
  plan.per = plan.start + kPlan;
  plan.band = plan.per + kPlan;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&qfull[s], 1);
      mbar_init(&pfull[s], 2);  // by each block
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 16);  // eight warps of each block
    }
    for (int b = 0; b < 4; ++b) mbar_init(&rbar[b], 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  make_plan<PASS>(p, plan, warp_sums);
  const uint32_t first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------- copies (both blocks) ------------------------------
    if (lane == 0) {
      const int bn2 = p.bn / 2;  // columns a copy brings
      const uint32_t bytes = kABytes + static_cast<uint32_t>(PASS == kWgrad ? 128 : bn2) * kL * 2;
      int stage = 0;
      uint32_t phase = 0;
      InFlight fly;
      bool ok = true;
      Walker<PASS, MT> walk(p, plan, first, step);
      Tile tile;
      while (ok && walk.next(tile)) {
        const int m0 = tile.m0 + rank * kM, c0 = tile.c0 + rank * (pair_columns(tile) / 2);
        const int nk = (tile.len + kL - 1) / kL;
        for (int kb = 0; kb < nk; ++kb) {
          if (!wait_phase<false>(&empty[stage], phase ^ 1u, p.ctrl, abort_flag)) { ok = false; break; }
          unsigned char* a = smem + stage * C::kStageBytes;
          unsigned char* b = a + kABytes;
          const bool partial = PASS == kWgrad && tile.len - kb * kL < kL;
          const uint32_t fb = partial ? mapa_shared(smem_u32(&qfull[stage]), static_cast<uint32_t>(rank))
                                      : mapa_shared(smem_u32(&full[stage]), 0);
          if (partial) mbar_arrive_expect_tx(&qfull[stage], bytes);
          else if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
          if (PASS == kWgrad) {
            const int l = tile.l0 + kb * kL;
            tma_load_2d_pair(a, &p.tmA, m0, l, fb);
            tma_load_2d_pair(a + kChunkBytes, &p.tmA, m0 + 64, l, fb);
            tma_load_2d_pair(b, &p.tmB, c0, l, fb);
            tma_load_2d_pair(b + kChunkBytes, &p.tmB, c0 + 64, l, fb);
          } else {
            if (PASS == kFwd) {
              tma_load_3d_pair(a, &p.tmA, kb * kL, m0, tile.e, fb);
            } else {
              tma_load_3d_pair(a, &p.tmA, m0, kb * kL, tile.e, fb);
              tma_load_3d_pair(a + kChunkBytes, &p.tmA, m0 + 64, kb * kL, tile.e, fb);
            }
            tma_load_2d_pair(b, &p.tmB, kb * kL, c0, fb);
          }
          fly.issue(stage, partial);
          if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        }
      }
      fly.land<C::kStages>(rank == 0 ? full : nullptr, qfull, p.ctrl);
    }
  } else if (warp == 1) {
    // ------------------------------- MMAs (even block) ---------------------------------
    if (rank == 0 && lane == 0) {
      const uint32_t major = (PASS == kFwd ? 0u : 1u << 15) | (PASS == kWgrad ? 1u << 16 : 0u);
      const uint32_t sa = smem_u32(smem), sb = sa + kABytes;  // of stage 0
      Ring<C::kStages, C::kStageBytes> ring{full, empty, PASS == kFwd ? sw128_kmajor_desc(sa) : sw128_mnmajor_desc(sa),
                                            PASS == kWgrad ? sw128_mnmajor_desc(sb) : sw128_kmajor_desc(sb), 0, 0u, 0u};
      int acc = 0;        // as in gemm_tc_kernel
      uint32_t uses = 0;
      bool ok = true;
      Walker<PASS, MT> walk(p, plan, first, step);
      Tile tile;
      while (ok && walk.next(tile)) {
        const int nk = (tile.len + kL - 1) / kL;
        if (nk == 0) continue;
        const uint32_t idesc = idesc_bf16_f32(MT, pair_columns(tile)) | major;
        const int left = tile.len - (nk - 1) * kL;
        const int parts = parts_of(nk);
        for (int i = 0; i < parts; ++i) {
          const bool last = i + 1 == parts;
          const int a = i ? acc ^ 1 : acc;
          const int n = parts == 1 ? nk : part_begin(nk, i + 1, parts) - part_begin(nk, i, parts);
          ok = wait_phase<true>(&tempty[a], ((uses >> a) & 1u) ^ 1u, p.ctrl, abort_flag);
          if (!ok) break;
          tc_fence_after();
          ok = mma_stages<PASS, true, 0>(ring, n, last ? (left + 15) / 16 : kL / 16, tmem_base + a * C::BN, idesc,
                                         last && left < kL ? pfull : nullptr, p.ctrl, abort_flag);
          if (!ok) break;
          mma_commit_pair(&tfull[a]);
          uses ^= 1u << a;
        }
        acc ^= 1;
      }
      mma_commit_pair(drain);  // every MMA done before the accumulators are freed
      wait_phase<false>(drain, 0, p.ctrl, nullptr);
    }
  } else if (warp == kPatchWarp) {
    if (PASS == kWgrad) {
      // ----------------------------- partial stages (both blocks) ----------------------
      int stage = 0;        // of the tile's first reduction steps
      uint32_t phases = 0;  // per stage: parity of its next partial use
      Walker<PASS, MT> walk(p, plan, first, step);
      Tile tile;
      while (walk.next(tile)) {
        const int nk = (tile.len + kL - 1) / kL;
        const int left = tile.len - (nk - 1) * kL;
        if (nk > 0 && left < kL) {
          const int at = (stage + nk - 1) % C::kStages;
          if (!warp_wait_phase<false>(&qfull[at], (phases >> at) & 1u, p.ctrl, abort_flag)) break;
          phases ^= 1u << at;
          zero_rows(smem + at * C::kStageBytes, 4, left, (left + 15) / 16 * 16);
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&pfull[at]), 0));
        }
        stage = (stage + nk) % C::kStages;
      }
    }
  } else {
    // ------------------------------- epilogue (both blocks) ----------------------------
    const int quarter = warp & 3;
    const uint32_t release0 = mapa_shared(smem_u32(&tempty[0]), 0), release1 = mapa_shared(smem_u32(&tempty[1]), 0);
    Group grp{(warp - 2) >> 2, nullptr, nullptr, nullptr, nullptr, 0, 0u, threadIdx.x % 128 == 64};
    grp.out = staging + grp.id * kGroupBytes<PASS, FULL>;
    grp.pre = grp.out + kOutBufs<PASS> * kChunk;
    grp.res = grp.pre + kChunk;
    grp.rbar = rbar + 2 * grp.id;
    int acc = 0;
    uint32_t uses = 0;
    bool failed = false;
    Walker<PASS, MT> walk(p, plan, first, step);
    Tile tile;
    while (walk.next(tile)) {
      const bool has = tile.len > 0;
      const uint32_t trow0 = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
      const uint32_t trow = trow0 + acc * C::BN;
      auto finished = [&](int a) {
        if (!failed && !wait_phase<true>(&tfull[a], (uses >> a) & 1u, p.ctrl, abort_flag)) failed = true;
        uses ^= 1u << a;
        __syncwarp();
        tc_fence_after();
      };
      auto ready = [&] {
        if (!has) return;
        finished(acc);
        for (int i = 1; i < parts_of((tile.len + kL - 1) / kL); ++i) {
          finished(acc ^ 1);
          constexpr int kWidth = kTaken<PASS, C::BN>;
          add_part<C::BN, 1>(trow, trow0 + (acc ^ 1) * C::BN, grp.id * kWidth, kWidth, 2 * kWidth, tile.ncols);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(acc ? release0 : release1);
        }
      };
      store_tile<PASS, C::BN, FULL>(p, tile, tile.m0 + rank * kM, trow, has ? 1 : 0, grp, ready, [&] {
        if (lane == 0) mbar_arrive_remote(acc ? release1 : release0);
      });
      if (has) acc ^= 1;
    }
    bulk_wait();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither block leaves while the pair's MMAs may still read its operands
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// ------------------------------- host ---------------------------------------------------
bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, uint32_t box0, uint32_t box1) {
  EncodeTiledFn fn = get_encode_tiled();
  if (!fn) return false;
  const cuuint64_t strides[2] = {dims[0] * 2, dims[0] * dims[1] * 2};
  const cuuint32_t box[3] = {box0, box1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a kernel's launches need to know of the device, found once: its shared memory limit is
// raised, and the clusters of each size that fit on the device at a time are counted (a cluster
// stays within a part of the chip, so fewer fit than SMs would allow; one too many would run
// after all the others).  KERN is a template argument so that each kernel keeps its own record.
template <auto KERN>
int units_on_device(int smem, int cluster, int num_sms) {
  static std::atomic<int> known[64][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::atomic<int>& mine = known[dev][cluster == 1 ? 0 : cluster == 2 ? 1 : cluster == 4 ? 2 : 3];
  int n = mine.load(std::memory_order_acquire);
  if (n) return n;
  if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
  n = num_sms;
  if (cluster > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms / cluster * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, KERN, &cfg) != cudaSuccess || n < 1) return 0;
    n = std::min(n, num_sms / cluster);
  }
  mine.store(n, std::memory_order_release);
  return n;
}

// Launch in clusters of `cluster` blocks (1: none), at most one block an SM.
template <auto KERN>
cudaError_t launch(const TcParams& p, int smem, int64_t tiles, int num_sms, int cluster, cudaStream_t st) {
  const int fit = units_on_device<KERN>(smem, cluster, num_sms);
  if (fit < 1) return cudaErrorInvalidConfiguration;
  const int64_t units = std::max<int64_t>(1, std::min<int64_t>(tiles, fit));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, KERN, p);
}

template <int PASS, int BN>
cudaError_t launch_split(const TcParams& p, int64_t tiles, int num_sms, int cluster, cudaStream_t st) {
  return launch<gemm_tc_kernel<PASS, BN, true, false>>(p, Cfg<PASS, BN, true, false>::kSmemBytes, tiles, num_sms, cluster,
                                                       st);
}
template <int PASS, int BN>
cudaError_t launch_tc(const TcParams& p, int64_t tiles, int num_sms, cudaStream_t st) {
  if constexpr (PASS == kFwd) {
    if (p.residual || p.preact)
      return launch<gemm_tc_kernel<PASS, BN, false, true>>(p, Cfg<PASS, BN, false, true>::kSmemBytes, tiles, num_sms, 1, st);
  }
  return launch<gemm_tc_kernel<PASS, BN, false, false>>(p, Cfg<PASS, BN, false, false>::kSmemBytes, tiles, num_sms, 1, st);
}
template <int PASS>
cudaError_t launch_pair(const TcParams& p, int64_t tiles, int num_sms, cudaStream_t st) {
  if constexpr (PASS == kFwd) {
    if (p.residual || p.preact)
      return launch<gemm_pair_kernel<PASS, true>>(p, PairCfg<PASS, true>::kSmemBytes, tiles, num_sms, 2, st);
  }
  return launch<gemm_pair_kernel<PASS, false>>(p, PairCfg<PASS, false>::kSmemBytes, tiles, num_sms, 2, st);
}
template <int PASS, int BN>
int split_units(int cluster, int num_sms) {
  return units_on_device<gemm_tc_kernel<PASS, BN, true, false>>(Cfg<PASS, BN, true, false>::kSmemBytes, cluster, num_sms);
}

template <int PASS>
cudaError_t launch_pass(const GemmArgs& a, cudaStream_t st) {
  TcParams p{};
  p.offsets = a.offsets;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.bias = a.bias;
  p.residual = static_cast<const __nv_bfloat16*>(a.residual);
  p.preact = static_cast<__nv_bfloat16*>(a.preact);
  p.R = a.R;
  p.M = PASS == kFwd ? a.N : a.K;
  p.C = a.N;
  p.L = PASS == kFwd ? a.K : a.N;
  p.E = a.E;
  p.act = a.act;
  p.ctrl = a.ctrl;
  const int64_t mt = (p.M + kM - 1) / kM;
  const int64_t per_group = (a.R + a.E - 1) / a.E;
  // Columns per tile.  Rows: enough for a group somewhat above the average in one tile (its
  // weights are then read once), in steps of 16, and of several groups at least 64, for those far
  // above it (288 experts of 1280 x 4096, 4096 rows: all in one group 186 us with tiles of 32
  // and 107 with 64; spread evenly 464, 465 and, with 128, 488).  wgrad: boxes of 64 output features.
  int bn;
  if (PASS == kWgrad) {
    bn = std::min(256, (a.N + 63) / 64 * 64);
  } else {
    const int64_t want = a.E == 1 ? per_group : per_group + per_group * 2 / 5 + 4;
    bn = static_cast<int>(std::min<int64_t>(256, (want + 15) / 16 * 16));
    if (a.E > 1) bn = std::max(bn, static_cast<int>(std::min<int64_t>(64, (a.R + 15) / 16 * 16)));
  }
  auto tiles_of = [&](int n) {  // at most
    const int64_t ct = PASS == kWgrad ? static_cast<int64_t>(a.E) * ((a.N + n - 1) / n)
                                      : (a.E == 1 ? (a.R + n - 1) / n : a.R / n + std::min<int64_t>(a.R, a.E));
    return ct * mt;
  };
  // Enough tall tiles for every pair of SMs, wide enough to be worth halving the copies
  const bool pair = bn >= 128 && p.M > kM && tiles_of(bn) >= 2 * a.num_sms;
  if (pair && PASS != kWgrad) bn = (bn + 31) / 32 * 32;
  if (pair && PASS == kWgrad) bn = 256;
  // Too few tiles for the SMs: narrower ones, then slices of the reduction over a cluster
  while (!pair && bn > 64 && tiles_of(bn) < a.num_sms) bn = std::max(64, bn / 2 / 64 * 64);
  const int64_t stages = ((PASS == kWgrad ? per_group : p.L) + kL - 1) / kL;
  // Blocks that share a tile.  In units of a stage's MMAs: a round of tiles takes its share of
  // the stages, two more where partial sums are exchanged, and three once for their last
  // exchange (4 x 4096 x 4096, 32 tiles of 64 stages: 24.0 us for one block a tile, 16.2 for two,
  // 12.9 for four, 19.9 for eight, which need a second round; 16 x 11264 x 4096, 88 tiles: 26.6
  // for one, 31.1 for two).
  int cluster = 1;
  if (bn <= 64) {
    int64_t best = 0;
    for (int c = 1; c <= 8 && c <= stages; c *= 2) {
      int units = a.num_sms;
      if (c > 1) {
        if constexpr (PASS != kWgrad) {
          units = bn <= 16 ? split_units<PASS, 16>(c, a.num_sms) : split_units<PASS, 64>(c, a.num_sms);
        } else {
          units = split_units<PASS, 64>(c, a.num_sms);
        }
        if (units < 1) return cudaErrorInvalidConfiguration;
      }
      const int64_t rounds = (tiles_of(bn) + units - 1) / units;
      const int64_t cost = rounds * ((stages + c - 1) / c + (c > 1 ? 2 : 0)) + (c > 1 ? 3 : 0);
      if (c == 1 || cost < best) {
        best = cost;
        cluster = c;
      }
    }
  }
  p.bn = bn;
  p.mt = FastDiv(static_cast<uint32_t>(pair ? (p.M + 2 * kM - 1) / (2 * kM) : mt));
  p.ct = FastDiv(static_cast<uint32_t>((a.N + bn - 1) / bn));
  p.ct_band = band_of(static_cast<int>(p.ct.d));
  const int64_t tiles = tiles_of(bn);

  const cuuint64_t dims_w[3] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.N), static_cast<cuuint64_t>(a.E)};
  const cuuint64_t dims_x[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(std::max<int64_t>(a.R, 1))};
  const cuuint64_t dims_y[2] = {static_cast<cuuint64_t>(a.N), static_cast<cuuint64_t>(std::max<int64_t>(a.R, 1))};
  const uint32_t box = static_cast<uint32_t>(pair ? bn / 2 : bn);  // rows a copy brings
  bool ok;
  if (PASS == kFwd) {
    ok = encode(&p.tmA, a.other, 3, dims_w, kL, kM) && encode(&p.tmB, a.rows, 2, dims_x, kL, box);
  } else if (PASS == kDgrad) {
    ok = encode(&p.tmA, a.other, 3, dims_w, 64, kL) && encode(&p.tmB, a.rows, 2, dims_y, kL, box);
  } else {
    // without rows only zeros are written: the maps then stand on `out` and copy nothing
    ok = encode(&p.tmA, a.R ? a.other : a.out, 2, dims_x, 64, kL) &&
         encode(&p.tmB, a.R ? a.rows : a.out, 2, dims_y, 64, kL);
  }
  // out as rows of M features; a chunk is 16 rows for the narrowest accumulators, else kCols
  const cuuint64_t dims_o[2] = {static_cast<cuuint64_t>(p.M),
                                static_cast<cuuint64_t>(PASS == kWgrad ? static_cast<int64_t>(a.E) * a.N : a.R)};
  const uint32_t chunk = bn <= 16 ? 16 : kCols;
  ok = ok && encode(&p.tmO, a.out, 2, dims_o, 64, chunk) &&
       (!a.residual || encode(&p.tmR, a.residual, 2, dims_o, 64, chunk)) &&
       (!a.preact || encode(&p.tmZ, a.preact, 2, dims_o, 64, chunk));
  if (!ok) return cudaErrorInvalidValue;
  if (pair) return launch_pair<PASS>(p, (tiles + 1) / 2, a.num_sms, st);
  if (cluster > 1) {
    if constexpr (PASS != kWgrad) {
      if (bn <= 16) return launch_split<PASS, 16>(p, tiles, a.num_sms, cluster, st);
    }
    return launch_split<PASS, 64>(p, tiles, a.num_sms, cluster, st);
  }
  if constexpr (PASS != kWgrad) {
    if (bn <= 16) return launch_tc<PASS, 16>(p, tiles, a.num_sms, st);
  }
  if (bn <= 64) return launch_tc<PASS, 64>(p, tiles, a.num_sms, st);
  if (bn <= 128) return launch_tc<PASS, 128>(p, tiles, a.num_sms, st);
  return launch_tc<PASS, 256>(p, tiles, a.num_sms, st);
}

}  // namespace

cudaError_t launch_gemm_bf16(const GemmArgs& a, cudaStream_t st) {
  switch (a.pass) {
    case kFwd: return launch_pass<kFwd>(a, st);
    case kDgrad: return launch_pass<kDgrad>(a, st);
    default: return launch_pass<kWgrad>(a, st);
  }
}

}  // namespace moe
