// Segment statistics of rows of vocabulary logits: the one pass over the logits that the
// distillation loss and the beam selection make.
//
// For each segment (1024 bf16 or 512 fp32 consecutive ids of a row): m = max z and
// sum exp((z - m)/T).  The bound is HBM: the logits are read once and 8 bytes are written per 2 KB.
// A warp holds a whole segment in registers, so the sum is taken relative to the segment's true
// maximum, without a running rescale, with one reduction pair per 32 elements of a lane.  The
// warps stream the (row, segment) items of all rows, so a row longer than a warp's share is split
// over many SMs and few rows still use the whole card.  64 warps per SM (32 registers) keep enough
// loads in flight without any in the code: 2048 rows of 151936 bf16 logits, 622 MB, 95 us, 6.5 TB/s.  A
// beam step over them takes 103 us; with the next item's loads issued ahead (48 registers, fewer warps) 110.
// With 32 warps it takes 121 instead of 105, each step waited for.
#include "rows.cuh"

namespace dh {
namespace {

constexpr int RS_THREADS = 256;

// The factor c = log2(e)/T is one float, so a row's sum has the error of a temperature that is off by
// 2^-24: up to 1e-7 in its logarithm, as much as the 2^x unit's own (5e-8 on average).  A second
// multiply-add by the rest of c takes that part away and leaves the unit's: the errors of random rows then
// are 0 to 7e-8 instead of -8e-8 to 1e-7, for 9 us more at 2048 rows of 151936 bf16 logits.

// Index: unsigned where the items' numbers fit, else long long (a 64-bit division per item costs as much
// as a third of its logits).
template <typename T, bool ALIGNED, typename Index>
__global__ void __launch_bounds__(RS_THREADS) k_row_stats(const T* __restrict__ logits, long long rs,
                                                          long long ws, int W, int vocab, float c, int n_seg,
                                                          Index n_items,
                                                          const float* __restrict__ score,
                                                          const int32_t* __restrict__ finished,
                                                          float2* __restrict__ seg) {
  constexpr int PER = Elem<T>::PER16;
  const int lane = threadIdx.x & 31;
  const Index nw = (Index)gridDim.x * (RS_THREADS / 32);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // only now: the kernel after this one reads the call's inputs as soon as it may start
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (Index g = (Index)blockIdx.x * (RS_THREADS / 32) + (threadIdx.x >> 5); g < n_items; g += nw) {
    const int row = (int)(g / (Index)n_seg), sgi = (int)(g - (Index)row * (Index)n_seg);
    if (score) {
      // a beam without candidates of its own: its logits are not read
      const float sc = __ldg(score + row);
      if (!(fabsf(sc) < INFINITY) || (finished && __ldg(finished + row) != 0)) continue;
    }
    const int rq = W == 1 ? row : row / W;
    const T* r = logits + rq * rs + (row - rq * W) * ws;
    uint4 u[ROW_SEG_VECS];
    const int id0 = sgi * row_seg<T>() + lane * PER;
#pragma unroll
    for (int v = 0; v < ROW_SEG_VECS; ++v) u[v] = row_vec<T, ALIGNED>(r, id0 + v * 32 * PER, vocab);
    const float2 p = segment_stats<T>(u, c);
    if (lane == 0) seg[g] = p;
  }
}

template <typename T>
cudaError_t run(const Ctx& c, const void* logits, long long rs, long long ws, int R, int W, int vocab,
                float temperature, const float* score, const int32_t* finished, float2* seg) {
  const int n_seg = (vocab + row_seg<T>() - 1) / row_seg<T>();
  const long long n_items = (long long)R * W * n_seg;
  const long long per_block = RS_THREADS / 32;
  const long long want = (n_items + per_block - 1) / per_block;
  const unsigned grid = (unsigned)(want < 8LL * c.num_sms ? want : 8LL * c.num_sms);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(RS_THREADS);
  cfg.stream = c.stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const float cf = (float)(1.4426950408889634 / (double)temperature);
  const bool aligned = rows_aligned(logits, rs, ws, R, W, (int)sizeof(T));
  prof_before("row_stats", c.stream);
  const T* z = static_cast<const T*>(logits);
  auto go = [&](auto* kernel, auto items) {
    return cudaLaunchKernelEx(&cfg, kernel, z, rs, ws, W, vocab, cf, n_seg, items, score, finished, seg);
  };
  // nw more than the last item's number still has to fit
  const bool narrow = n_items < 0x7F000000LL;
  const cudaError_t e =
      narrow ? (aligned ? go(k_row_stats<T, true, unsigned>, (unsigned)n_items)
                        : go(k_row_stats<T, false, unsigned>, (unsigned)n_items))
             : (aligned ? go(k_row_stats<T, true, long long>, n_items) : go(k_row_stats<T, false, long long>, n_items));
  prof_after(c.stream);
  return e;
}

}  // namespace

int row_segments(int vocab, int dtype) {
  const int seg = dtype == DH_BF16 ? row_seg<__nv_bfloat16>() : row_seg<float>();
  return (vocab + seg - 1) / seg;
}

// Whether every row [r][w] starts on 16 bytes.
bool rows_aligned(const void* logits, long long rs, long long ws, int R, int W, int elem) {
  return (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 && (R == 1 || rs * elem % 16 == 0) &&
         (W == 1 || ws * elem % 16 == 0);
}

cudaError_t launch_row_stats(const Ctx& c, const void* logits, long long rs, long long ws, int R, int W, int vocab,
                             int dtype, float temperature, const float* score, const int32_t* finished, float2* seg) {
  return dtype == DH_BF16 ? run<__nv_bfloat16>(c, logits, rs, ws, R, W, vocab, temperature, score, finished, seg)
                          : run<float>(c, logits, rs, ws, R, W, vocab, temperature, score, finished, seg);
}

}  // namespace dh
