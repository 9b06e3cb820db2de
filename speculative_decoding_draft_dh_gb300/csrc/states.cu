// Moving the drafter's states after a selection: slot j of a request takes its slot idx[j]
// (definition at dh_reorder_states in dh.h).
//
// Nothing is computed, so the bound is HBM: each source that is needed read once, each target
// written once.  A thread owns one column, the same few bytes (16 where the layout allows) of every
// slot of a request: it loads the column's M sources and then stores them.  No other thread touches
// the column, so in place needs no more than a thread's own order (all loads before the first
// store) and no second buffer; a source that several targets share is fetched from HBM once, its
// loads being issued together.
// 8 requests of 8 beams, 2.35 GB in caches of up to 4096 positions: 336 us, 7.0 TB/s (the copy's rate);
// the accepted paths of 64 trees, 12.6 MB: 6 us, a chain of two loads and the launch.
//   k_reorder:          separate source and target: batches of 8 slots in registers.
//   k_reorder_inplace:  up to 16 moves in registers; more are staged in the block's shared memory,
//                       as many columns at a time as fit.  Slots that stay where they are cost
//                       nothing.
// In place, caches of 1.07 GB, bf16: 8 beams 314 us (223 for the bytes of the slots that move: the loaded
// slots take 80 registers, with spills), 24 beams, staged, 865 us (256: 128 KB per block, so one block per
// SM).  With lengths, positions innermost (a transposed cache) are moved one element at a time: 1285 us and
// 5220; put the positions before the contiguous part.
#include "operators.cuh"

namespace dh {
namespace {

constexpr int RO_THREADS = 256;
constexpr int RO_BATCH = 8;
constexpr int RO_REGS = 16;               // in-place moves that stay in registers
constexpr int RO_STAGE = 128 * 1024;      // bytes of staging for more

template <int V> struct Unit;
template <> struct Unit<16> { using T = uint4; };
template <> struct Unit<8> { using T = uint2; };
template <> struct Unit<4> { using T = uint32_t; };
template <> struct Unit<2> { using T = unsigned short; };
template <> struct Unit<1> { using T = unsigned char; };

// Where a block stands: tensor slice (a, r) and its first column.
struct Place {
  long long a;
  int r;
  uint32_t col0;
};
__device__ __forceinline__ Place place(const ReorderArgs& p, uint32_t blocks_per_slice) {
  const uint32_t slice = blockIdx.x / blocks_per_slice;
  Place q;
  q.a = slice / (uint32_t)p.R;
  q.r = (int)(slice - (uint32_t)q.a * (uint32_t)p.R);
  q.col0 = (blockIdx.x - slice * blocks_per_slice) * RO_THREADS;
  return q;
}

// Offsets of column `col` = (h, t, v) in source and target; false past the last or the length.
__device__ __forceinline__ bool column(const ReorderArgs& p, uint32_t col, uint32_t cols, uint32_t per_t, int V,
                                       int len, long long* so, long long* dso) {
  if (col >= cols) return false;
  const uint32_t x = col / per_t, v = col - x * per_t;
  const uint32_t h = x / (uint32_t)p.T, t = x - h * (uint32_t)p.T;
  if ((int)t >= len) return false;
  *so = h * p.ss[3] + t * p.ss[4] + (long long)v * V;
  *dso = h * p.ds[3] + t * p.ds[4] + (long long)v * V;
  return true;
}

// Source slot and target slot of move j of request r; false where there is none.
__device__ __forceinline__ bool move_of(const ReorderArgs& p, int r, int j, int sb, int db, int* from, int* to) {
  const int i = __ldg(p.idx + (long long)r * p.M + j);
  const long long f = (long long)sb + i, t = (long long)db + j;
  *from = (int)f;
  *to = (int)t;
  return i >= 0 && f >= 0 && f < p.src_slots && t >= 0 && t < p.dst_slots;
}

template <int V>
__global__ void __launch_bounds__(RO_THREADS) k_reorder(ReorderArgs p, uint32_t blocks_per_slice, uint32_t cols,
                                                        uint32_t per_t) {
  using T = typename Unit<V>::T;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Place q = place(p, blocks_per_slice);
  const int len = p.lengths ? min(max(__ldg(p.lengths + q.r), 0), p.T) : p.T;
  const int sb = p.src_base ? __ldg(p.src_base + q.r) : 0, db = p.dst_base ? __ldg(p.dst_base + q.r) : 0;
  long long so, dso;
  if (!column(p, q.col0 + threadIdx.x, cols, per_t, V, len, &so, &dso)) return;
  const char* src = p.src + q.a * p.ss[0] + q.r * p.ss[1] + so;
  char* dst = p.dst + q.a * p.ds[0] + q.r * p.ds[1] + dso;
  for (int j0 = 0; j0 < p.M; j0 += RO_BATCH) {
    T x[RO_BATCH];
    int to[RO_BATCH];
#pragma unroll
    for (int b = 0; b < RO_BATCH; ++b) {
      int from = 0, t = 0;
      const bool ok = j0 + b < p.M && move_of(p, q.r, j0 + b, sb, db, &from, &t);
      to[b] = ok ? t : -1;
      if (ok) x[b] = __ldg(reinterpret_cast<const T*>(src + from * p.ss[2]));
    }
#pragma unroll
    for (int b = 0; b < RO_BATCH; ++b)
      if (to[b] >= 0) *reinterpret_cast<T*>(dst + to[b] * p.ds[2]) = x[b];
  }
}

template <int V>
__global__ void __launch_bounds__(RO_THREADS) k_reorder_inplace(ReorderArgs p, uint32_t blocks_per_slice,
                                                                uint32_t cols, uint32_t per_t) {
  using T = typename Unit<V>::T;
  extern __shared__ __align__(16) unsigned char stage[];
  __shared__ int s_from[DH_MAX_SLOTS], s_to[DH_MAX_SLOTS];
  __shared__ int s_n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Place q = place(p, blocks_per_slice);
  const int len = p.lengths ? min(max(__ldg(p.lengths + q.r), 0), p.T) : p.T;
  const int sb = p.src_base ? __ldg(p.src_base + q.r) : 0, db = p.dst_base ? __ldg(p.dst_base + q.r) : 0;
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < p.M; j += RO_THREADS) {
    int from, to;
    if (move_of(p, q.r, j, sb, db, &from, &to) && from != to) {
      const int at = atomicAdd(&s_n, 1);  // the moves' order does not matter: all loads come first
      s_from[at] = from;
      s_to[at] = to;
    }
  }
  __syncthreads();
  const int n = s_n;
  if (n == 0) return;
  char* base = p.dst + q.a * p.ds[0] + q.r * p.ds[1];
  if (n <= RO_REGS) {
    long long so, dso;
    if (!column(p, q.col0 + threadIdx.x, cols, per_t, V, len, &so, &dso)) return;
    T x[RO_REGS];
#pragma unroll
    for (int b = 0; b < RO_REGS; ++b)
      if (b < n) x[b] = *reinterpret_cast<const T*>(base + dso + s_from[b] * p.ds[2]);
#pragma unroll
    for (int b = 0; b < RO_REGS; ++b)
      if (b < n) *reinterpret_cast<T*>(base + dso + s_to[b] * p.ds[2]) = x[b];
    return;
  }
  // columns [c0, c0 + width) at a time, one per thread: stage[move][column]
  T* st = reinterpret_cast<T*>(stage);
  const int fit = RO_STAGE / (int)sizeof(T) / n;
  const int width = fit < RO_THREADS ? fit : RO_THREADS;
  for (int c0 = 0; c0 < RO_THREADS; c0 += width) {
    const int c = c0 + (int)threadIdx.x;
    long long so, dso;
    if ((int)threadIdx.x >= width || c >= RO_THREADS || !column(p, q.col0 + c, cols, per_t, V, len, &so, &dso))
      continue;
    // a thread's own places in the staging, so no barrier
    for (int b = 0; b < n; ++b)
      st[b * width + threadIdx.x] = *reinterpret_cast<const T*>(base + dso + s_from[b] * p.ds[2]);
    for (int b = 0; b < n; ++b) *reinterpret_cast<T*>(base + dso + s_to[b] * p.ds[2]) = st[b * width + threadIdx.x];
  }
}

template <int V>
cudaError_t run(const Ctx& c, const ReorderArgs& a) {
  const uint32_t per_t = (uint32_t)(a.unit / V);
  const uint32_t cols = (uint32_t)((long long)a.H * a.T * per_t);  // < 2^31: checked by the caller
  const uint32_t bps = (cols + RO_THREADS - 1) / RO_THREADS;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.A * a.R * bps));  // < 2^31: checked by the caller
  cfg.blockDim = dim3(RO_THREADS);
  cfg.stream = c.stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e;
  prof_before("reorder", c.stream);
  if (a.in_place) {
    cfg.dynamicSmemBytes = a.M > RO_REGS ? RO_STAGE : 0;
    static unsigned long long done = 0;
    e = a.M > RO_REGS ? allow_max_smem(k_reorder_inplace<V>, c.device, &done) : cudaSuccess;
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, k_reorder_inplace<V>, a, bps, cols, per_t);
  } else {
    e = cudaLaunchKernelEx(&cfg, k_reorder<V>, a, bps, cols, per_t);
  }
  prof_after(c.stream);
  return e;
}

}  // namespace

// Widest power of two (up to 16 bytes) that every address of the copy is a multiple of.
int reorder_vector(const ReorderArgs& a) {
  uintptr_t bits = reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst) | (uintptr_t)a.unit;
  const int n[5] = {a.A, a.R, 2, a.H, a.T};
  for (int i = 0; i < 5; ++i)
    if (n[i] > 1) bits |= (uintptr_t)a.ss[i] | (uintptr_t)a.ds[i];
  int v = 16;
  while (bits & (uintptr_t)(v - 1)) v >>= 1;
  return v;
}

// Threads' columns per (a, r) slice and blocks of the launch (the caller checks their limits).
long long reorder_columns(const ReorderArgs& a) { return (long long)a.H * a.T * (a.unit / reorder_vector(a)); }
long long reorder_blocks(const ReorderArgs& a) {
  return (long long)a.A * a.R * ((reorder_columns(a) + RO_THREADS - 1) / RO_THREADS);
}

cudaError_t launch_reorder(const Ctx& c, const ReorderArgs& a) {
  switch (reorder_vector(a)) {
    case 16: return run<16>(c, a);
    case 8: return run<8>(c, a);
    case 4: return run<4>(c, a);
    case 2: return run<2>(c, a);
    default: return run<1>(c, a);
  }
}

}  // namespace dh
