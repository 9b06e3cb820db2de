// Layer norm over the last dimension, and its gradients (definitions at dh_layer_norm and
// dh_layer_norm_backward in dh.h).
//
// The bound is HBM: a row is read once and written once.  A row belongs to a group of threads, a vector of 16 bytes
// each or up to four; a block's groups walk over rows of their own, with the next rows on their way in shared memory
// while the present one is reduced in registers.  Once the memory is kept busy, the instructions count: they are
// packed in pairs, and the parameters wait in shared memory as fp32.  32768 rows of 5120 bf16: forward 102 us
// (671 MB, 6.6 TB/s), backward 173 (1.0 GB, 5.8 TB/s).  (The next rows in registers instead: 154 to 215 and 312 to 587;
// the parameters by way of L1: up to 313 backward.)
// Forward: the mean first, then the sums of x - mean and of its square, so that the variance loses nothing to a
// mean far from 0 (the two-pass form with the correction of Chan, Golub and LeVeque).
// Backward: with xhat = (x - mean) rstd and h = g w,
//   dx = rstd (h - mean(h) - xhat mean(h xhat)),   dw = sum_n g xhat,   db = sum_n g.
// A thread keeps its columns over all rows that its group walks, so dw and db are summed in its registers;
// blocks leave their sums in the workspace and a second kernel adds them in order.
// Rows of more than NM_HELD columns are read again for each step instead, by k_norm_wide and
// k_norm_backward_wide, and k_norm_columns sums their dw and db (10000 rows of 12288 bf16: 214 us and 433).
#include <mutex>
#include <type_traits>
#include <utility>
#include <vector>

#include "layers.cuh"
#include "rows.cuh"

namespace dh {
namespace {

constexpr int NM_HELD = 8192;  // columns of a row that registers hold

// Sums of a and b over the block, every thread gets them.  `turn` alternates, so that one barrier per call is
// enough.
__device__ __forceinline__ float2 block_sum(float a, float b, float2 (*sh)[32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sh[turn][warp] = make_float2(a, b);
  __syncthreads();
  float2 s = lane < warps ? sh[turn][lane] : make_float2(0.f, 0.f);
  turn ^= 1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
    s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
  }
  return s;
}

// One step of a reduction of several values at once: a lane keeps one of two, hands the other to the lane across,
// and takes that lane's share of what it keeps, so that K values cost K/2 + K/4 + ... exchanges.
__device__ __forceinline__ float fold(float low, float high, int o) {
  const bool up = threadIdx.x & o;
  return (up ? high : low) + __shfl_xor_sync(0xFFFFFFFFu, up ? low : high, o);
}

// Mean (as mean0 + delta) and 1 / sqrt(variance + eps) from the second pass's sums.
struct Moments {
  float mean0, delta, rstd;
};
__device__ __forceinline__ Moments moments(float mean0, float2 q, float inv_d, float eps) {
  const float delta = q.x * inv_d;
  float var = (q.y - q.x * delta) * inv_d;
  if (var < 0.f) var = 0.f;  // a NaN stays
  return {mean0, delta, 1.f / sqrtf(var + eps)};
}

// Rows on their way: SLOTS rows in shared memory.  A thread copies its own vectors by cp.async and reads them itself,
// so that no barrier is needed: 16 bytes each (VEC) or 4 (fp32 rows of any alignment).  Of bf16 rows off 16 bytes a
// warp copies the 16-byte words that hold its columns, and a thread reads its elements from there (20000 rows of 8191
// forward 171 us, backward 335; loaded element by element when they are used 283 and 412).
template <typename T, bool VEC, int NV>
struct Ring {
  using C = Cols<T, VEC, NV>;
  static constexpr bool WORDS = !VEC && sizeof(T) == 2;
  static constexpr int COPIES = VEC ? NV : NV * C::PER;  // of a thread and row
  static constexpr int STEP = VEC ? 32 * C::PER : 32;    // columns between them
  static constexpr int REGION = NV * 512 + (WORDS ? 16 : 0);  // bytes of a warp
  uint32_t mine;  // this thread's place in slot 0, a shared-memory address
  uint32_t slot;  // bytes of a slot
  int held;       // copies within the row (WORDS: columns of the warp)
  int first;      // this thread's (WORDS: its warp's) first column, 0 where it has none
  __device__ __forceinline__ Ring(void* smem, int me, int d)
      : mine((uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * REGION + (threadIdx.x & 31) * 16),
        slot(blockDim.x / 32 * REGION) {
    const int at = WORDS ? (me >> 5) * C::WARP : C::col(me, 0, 0);
    held = WORDS ? min(max(d - at, 0), C::WARP) : min(max((d - at + STEP - 1) / STEP, 0), COPIES);
    first = held ? at : 0;
  }
  static constexpr __host__ __device__ size_t bytes(int threads) { return (size_t)(threads / 32) * REGION; }
  __device__ __forceinline__ static void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  }
  // A row on its way to slot s (`on`: there is one), from its column `first` on.  A group of copies.
  __device__ __forceinline__ void fetch(const T* mine_of_row, bool on, int s) const {
    const uint32_t to = mine + s * slot;
    if constexpr (WORDS) {
      __syncwarp();  // the slot has been read
      if (on && held) {
        const int before = (int)(reinterpret_cast<uintptr_t>(mine_of_row) & 15u), lane = threadIdx.x & 31;
        const char* word = reinterpret_cast<const char*>(mine_of_row) - before;
        const int end = before + held * 2;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if ((lane + 32 * k) * 16 < end) copy16(to + k * 512, word + (lane + 32 * k) * 16);
        if (lane == 0 && NV * 512 < end) copy16(to + NV * 512, word + NV * 512);
      }
    } else if (on) {
#pragma unroll
      for (int k = 0; k < COPIES; ++k) {
        if constexpr (VEC) {
          // past the row's end: zeros, and the address is not used
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + k * 512),
                       "l"(mine_of_row + (k < held ? k * STEP : 0)), "r"(k < held ? 16 : 0)
                       : "memory");
        } else {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + (k / 4) * 512 + (k % 4) * 4),
                       "l"(mine_of_row + (k < held ? k * STEP : 0)), "r"(k < held ? 4 : 0)
                       : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // Waits for this thread's copies (WORDS: its warp's), up to the LATER youngest groups.
  template <int LATER>
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory");
    if constexpr (WORDS) __syncwarp();
  }
  // Vector v of the row in slot s.  WHOLE: the warp's columns all lie within the row.
  template <bool WHOLE = false>
  __device__ __forceinline__ uint4 get(const T* row, int s, int v) const {
    if constexpr (WORDS) {
      const int lane = threadIdx.x & 31;
      const uint32_t at = mine + s * slot - lane * 16 + (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < C::PER; ++e) {
        const int i = (v * C::PER + e) * 32 + lane;
        if (WHOLE || i < held) {
          unsigned short x;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at + i * 2) : "memory");
          w[e / 2] |= (uint32_t)x << (16 * (e & 1));
        }
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint4 u;
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                   : "r"(mine + s * slot + v * 512)
                   : "memory");
      return u;
    }
  }
};

// The elements of a vector in pairs.
template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& u, f32x2* z) {
  float x[Elem<T>::PER16];
  Elem<T>::unpack(u, x);
#pragma unroll
  for (int q = 0; q < Elem<T>::PER16 / 2; ++q) z[q] = pack2(x[2 * q], x[2 * q + 1]);
}
// The parameters of a thread's columns, 0 past the row's end.
template <typename T, typename P, bool VEC, int NV>
__device__ __forceinline__ void load_pairs(f32x2* w, const P* p, int thread, int v, int d) {
  using C = Cols<T, VEC, NV>;
  constexpr int PER = C::PER, PP = Elem<P>::PER16;
  float t[PER];
  if constexpr (VEC) {
    const int id = C::col(thread, v, 0);
#pragma unroll
    for (int q = 0; q < PER / PP; ++q) {
      const uint4 u = id < d ? __ldg(reinterpret_cast<const uint4*>(p + id) + q) : make_uint4(0u, 0u, 0u, 0u);
      Elem<P>::unpack(u, t + q * PP);
    }
  } else {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int id = C::col(thread, v, e);
      t[e] = id < d ? Elem<P>::to_f(p[id]) : 0.f;
    }
  }
#pragma unroll
  for (int e = 0; e < PER / 2; ++e) w[e] = pack2(t[2 * e], t[2 * e + 1]);
}
// Parameters in shared memory, as fp32 in the order in which the threads read them: each warp's vectors v, and of
// them the first four columns of all lanes before the other four (bank conflicts otherwise).
template <typename T, typename P, bool VEC, int NV>
struct SharedParams {
  using C = Cols<T, VEC, NV>;
  static constexpr int PER = C::PER;
  float* p;
  static constexpr __host__ __device__ size_t bytes(int width) { return (size_t)width * NV * PER * sizeof(float); }
  __device__ __forceinline__ explicit SharedParams(void* smem) : p(static_cast<float*>(smem)) {}
  __device__ __forceinline__ static int place(int col) {
    if (!VEC || PER == 4) return col;
    return (col & ~255) + ((col >> 3) & 31) * 4 + (col & 3) + ((col & 4) << 5);
  }
  __device__ __forceinline__ void fill(const P* src, int width, int d) const {
    if constexpr (VEC) {
      constexpr int PP = Elem<P>::PER16;
#pragma unroll 4
      for (int i = threadIdx.x * PP; i < width * NV * PER; i += blockDim.x * PP) {
        float t[PP];
        Elem<P>::unpack(i < d ? __ldg(reinterpret_cast<const uint4*>(src + i)) : make_uint4(0u, 0u, 0u, 0u), t);
#pragma unroll
        for (int h = 0; h < PP; h += 4)
          *reinterpret_cast<float4*>(p + place(i + h)) = make_float4(t[h], t[h + 1], t[h + 2], t[h + 3]);
      }
    } else {
#pragma unroll 4
      for (int i = threadIdx.x; i < width * NV * PER; i += blockDim.x) p[i] = i < d ? Elem<P>::to_f(src[i]) : 0.f;
    }
  }
  // The columns of vector v, in pairs.
  __device__ __forceinline__ void pairs(f32x2* w, int thread, int v) const {
    if constexpr (VEC) {
      const float* q = p + (thread >> 5) * C::WARP + v * 32 * PER + (thread & 31) * 4;
#pragma unroll
      for (int h = 0; h < PER / 4; ++h) {
        const float4 t = *reinterpret_cast<const float4*>(q + h * 128);
        w[2 * h] = pack2(t.x, t.y);
        w[2 * h + 1] = pack2(t.z, t.w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < PER; e += 2) w[e / 2] = pack2(p[C::col(thread, v, e)], p[C::col(thread, v, e + 1)]);
    }
  }
};
// Each rounded once to T.
template <typename T>
__device__ __forceinline__ uint4 round_pairs(const f32x2* z) {
  float x[Elem<T>::PER16];
#pragma unroll
  for (int q = 0; q < Elem<T>::PER16 / 2; ++q) unpack2(z[q], x[2 * q], x[2 * q + 1]);
  return round_vec<T>(x);
}
__device__ __forceinline__ f32x2 both(float x) { return pack2(x, x); }
__device__ __forceinline__ float half_of(f32x2 v, int high) {
  float a, b;
  unpack2(v, a, b);
  return high ? b : a;
}
__device__ __forceinline__ float pair_sum(f32x2 v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}

constexpr int NF_STAGES = 3;  // 32768 rows of 5120 bf16: 103 us, as with 2, 107 with 4
constexpr int NF_WARPS = 16;  // of a row, at most
// Registers of a thread with NV vectors.  With four, NF_TIGHT where they let more groups run (32768 rows of 5120: 4
// groups 102 us, 3 with 128 registers 106), else 128 (20000 rows of 8192: 2 groups of either kind 104 and 111).
constexpr int norm_regs(int nv) { return nv == 1 ? 64 : nv == 2 ? 80 : 128; }
constexpr int NF_TIGHT = 96;
// Threads of a block that have an SM's registers to themselves: a quarter of them to each four warps' first one.
constexpr int threads_by_regs(int regs) {
  return 65536 / 4 / 32 / regs * 128 < 1024 ? 65536 / 4 / 32 / regs * 128 : 1024;
}

// How a row ends: with a whole warp, within a warp that has eight elements of each thread or more (or is the only
// one, so that its c is no further out than the row's own deviations allow), or within a warp that has less.
enum RowEnd { WHOLE, LONG, SHORT };

// A block holds blockDim / width groups of `width` threads, each of which walks over rows of its own; the groups
// share the parameters (SHARED: in shared memory).  Barriers are a group's.
// A warp's sums are about the mean c of its threads' first eight elements each, the row's about the mean of up to
// four warps' means (the formulas of Chan, Golub and LeVeque).  Of what is joined one part in four or more enters
// the value that it is joined about, so the squares add up to about four times those about the mean at most, and
// nothing is lost to a mean far from 0 or to outliers, wherever they stand.  (About the mean of a single thread's
// elements they add up to d / 8 times an outlier's, which then cancels.)  Of means only differences and halves are
// added up: equal elements have no deviation at all.
// x - c, which the result is taken from, is rounded by 2^-24 |c|: that of an outlier's 256th part, less than the
// mean's own error allows.  But a warp that the row ends in may have less than those eight of each thread, and c is
// mostly an outlier's: its result is taken from x itself (a choice that costs 32768 rows of 5120 bf16 8 us of 110).
// Warps and vectors that lie within the row are read and summed without masks in rows off 16 bytes (20000 rows of
// 8191 bf16 166 us, 200 with masks, 182 with those of the last warp only; of 2047 42 and 51).
template <typename T, typename P, int NV, bool VEC, RowEnd END, bool SHARED, int REGS>
__global__ void __maxnreg__(REGS) k_norm(NormArgs a, int width) {
  using C = Cols<T, VEC, NV>;
  using S = SharedParams<T, P, VEC, NV>;
  constexpr int PER = C::PER, HALF = PER / 2;
  constexpr int REF = PER == 4 && NV > 1 ? 2 : 1;  // vectors whose mean a warp's sums are about
  extern __shared__ __align__(16) unsigned char norm_smem[];
  __shared__ __align__(16) float sh[2][32][4];  // of a warp: sum of x - c, c, sum of (x - c)^2
  const int group = threadIdx.x / width, groups = blockDim.x / width, me = threadIdx.x - group * width;
  const int warp = me >> 5, lane = me & 31, warps = width >> 5, warp0 = (threadIdx.x >> 5) - warp;
  const float inv_d = 1.f / (float)a.d;
  // elements of this thread's first vectors, of this thread, and of the warp whose sums this lane joins (lanes `span`
  // apart the same)
  int span = 1;
  while (span < warps) span *= 2;
  const int peer = lane & (span - 1);
  int first = 0, mine = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      mine += C::col(me, v, e) < a.d;
      if (v < REF) first = mine;
    }
  const float inv_first = first ? 1.f / (float)first : 0.f;
  const bool whole = (warp + 1) * C::WARP <= a.d;
  const int inside = (a.d - warp * C::WARP) / (32 * PER);  // vectors of the warp that lie within the row
  const bool empty = __any_sync(0xFFFFFFFFu, first == 0);  // the row ends within the warp
  const float their_count = (float)min(max(a.d - peer * C::WARP, 0), C::WARP);
  int turn = 0;
  const S w_shared(norm_smem), b_shared(norm_smem + S::bytes(width));
  const Ring<T, VEC, NV> ring(norm_smem + (SHARED ? 2 * S::bytes(width) : 0), me, a.d);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned rows = a.N, step = gridDim.x * groups;
  unsigned n = blockIdx.x * groups + group;
  const long long x_step = step * a.ld, y_step = step * a.y_ld;
  const T* row = static_cast<const T*>(a.x) + n * a.ld;
  const T* next = row + ring.first;  // the next row to fetch
  T* out = static_cast<T*>(a.y) + n * a.y_ld;
#pragma unroll
  for (int s = 0; s < NF_STAGES - 1; ++s) {
    ring.fetch(next, n + s * step < rows, s);
    next += x_step;
  }
  if constexpr (SHARED) {
    if (a.weight) w_shared.fill(static_cast<const P*>(a.weight), width, a.d);
    if (a.bias) b_shared.fill(static_cast<const P*>(a.bias), width, a.d);
    __syncthreads();
  }
  int stage = 0;
  for (; n < rows; n += step) {
    f32x2 z[NV][HALF];
    ring.template wait<NF_STAGES - 2>();
    // the row to registers, the mean c of the warp's first vectors, and the sums of x - c and of its square
    float c;
    f32x2 d1[2] = {0, 0}, d2[2] = {0, 0};
    auto take = [&](auto whole_warp) {
      constexpr bool W = decltype(whole_warp)::value;
      // (vectors that lie within the row need no masks)
      auto get = [&](int v) {
        if (W || VEC || v < inside) unpack_pairs<T>(ring.template get<true>(row, stage, v), z[v]);
        else unpack_pairs<T>(ring.template get<false>(row, stage, v), z[v]);
      };
#pragma unroll
      for (int v = 0; v < REF; ++v) get(v);
      // past the row's end the elements are 0
      f32x2 f = add2(z[0][0], z[0][1]);
      if constexpr (HALF == 4) f = add2(f, add2(z[0][2], z[0][3]));
      else if constexpr (REF == 2) f = add2(f, add2(z[1][0], z[1][1]));
      c = pair_sum(f) * inv_first;
      if (!W && empty) {
        const float other = __shfl_sync(0xFFFFFFFFu, c, 0);
        if (first == 0) c = other;
      }
      // (halves, so that equal ones stay what they are; each step while other loads are on their way)
      auto mix = [&](int o) {
        c *= 0.5f;
        c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
      };
      mix(16);
#pragma unroll
      for (int v = REF; v < NV; ++v) {
        get(v);
        mix(16 >> (v - REF + 1));
      }
      ring.fetch(next, n + (NF_STAGES - 1) * step < rows, stage == 0 ? NF_STAGES - 1 : stage - 1);
#pragma unroll
      for (int o = 16 >> (NV - REF + 1); o > 0; o >>= 1) mix(o);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        // and count for nothing
        const f32x2 shift = both(W || !VEC || v * PER < mine ? -c : 0.f);
        auto terms = [&](auto masked) {
#pragma unroll
          for (int e = 0; e < HALF; ++e) {
            f32x2 t = add2(z[v][e], shift);
            if constexpr (decltype(masked)::value) {
              float p, q;
              unpack2(t, p, q);
              t = pack2(v * PER + 2 * e < mine ? p : 0.f, v * PER + 2 * e + 1 < mine ? q : 0.f);
            }
            if constexpr (END != SHORT || VEC || W) z[v][e] = t;
            d1[e & 1] = add2(d1[e & 1], t);
            d2[e & 1] = fma2(t, t, d2[e & 1]);
          }
        };
        if (W || VEC || v < inside) terms(std::false_type{});
        else if (v == inside) terms(std::true_type{});
      }
    };
    if (END == WHOLE || (!VEC && whole)) take(std::true_type{});
    else if constexpr (END != WHOLE) take(std::false_type{});
    float own = c;  // what has been taken from z, or will be
    float part = fold(pair_sum(add2(d1[0], d1[1])), pair_sum(add2(d2[0], d2[1])), 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
    if (warps > 1) {
      // lanes 0 and 16 have the warp's sums
      if ((lane & 15) == 0) sh[turn][warp0 + warp][lane >> 3] = part;
      if (lane == 1) sh[turn][warp0 + warp][1] = c;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(width) : "memory");
      const float* q = sh[turn][warp0 + (peer < warps ? peer : 0)];
      // means of four of the warps without the last, which may have few columns
      auto mean_of = [&](int w) {
        const float2 t = *reinterpret_cast<const float2*>(sh[turn][warp0 + w]);
        return fmaf(t.x, 1.f / C::WARP, t.y);
      };
      const int most = warps - 1;
      c = mean_of(0);
      c += 0.25f * ((mean_of(most / 4) - c) + (mean_of(most / 2) - c) + (mean_of(most * 3 / 4) - c));
      part = 0.f;
      if (peer < warps) {
        const float g = q[1] - c, k = their_count * g;
        part = lane < 16 ? q[0] + k : fmaf(g, fmaf(2.f, q[0], k), q[2]);
      }
      turn ^= 1;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
        if (o < span) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
    }
    const float sum1 = __shfl_sync(0xFFFFFFFFu, part, 0), sum2 = __shfl_sync(0xFFFFFFFFu, part, 16);
    const float delta = sum1 * inv_d;
    float var = (sum2 - sum1 * delta) * inv_d;
    if (var < 0.f) var = 0.f;  // a NaN stays
    const float rs = 1.f / sqrtf(var + a.eps);
    // the mean, rounded, and what that leaves out
    const float mean = c + delta, rest = (c - mean) + delta;  // rounded, and what that leaves out
    if (a.stats_out && me == 0) a.stats_out[n] = make_float2(mean, rs);
    if (END == SHORT && !whole) {
      // (the row's slot is filled again in the next round)
      own = mean;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if constexpr (VEC) unpack_pairs<T>(ring.get(row, stage, v), z[v]);
#pragma unroll
        for (int e = 0; e < HALF; ++e) z[v][e] = add2(z[v][e], both(-mean));
      }
    }
    const f32x2 rstd = both(rs), back = both(((own - mean) - rest) * rs);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      f32x2 w[HALF], b[HALF];
      if (a.weight) {
        if constexpr (SHARED) w_shared.pairs(w, me, v);
        else load_pairs<T, P, VEC, NV>(w, static_cast<const P*>(a.weight), me, v, a.d);
      }
      if (a.bias) {
        if constexpr (SHARED) b_shared.pairs(b, me, v);
        else load_pairs<T, P, VEC, NV>(b, static_cast<const P*>(a.bias), me, v, a.d);
      }
#pragma unroll
      for (int e = 0; e < HALF; ++e) {
        f32x2 o = fma2(z[v][e], rstd, back);
        if (a.weight) o = a.bias ? fma2(o, w[e], b[e]) : mul2(o, w[e]);
        else if (a.bias) o = add2(o, b[e]);
        z[v][e] = o;
      }
      C::store(out, me, v, a.d, round_pairs<T>(z[v]));
    }
    out += y_step;
    next += x_step;
    row += x_step;
    stage = stage + 1 == NF_STAGES ? 0 : stage + 1;
  }
}

constexpr int NB_REGS = 128, NB_THREADS = 65536 / NB_REGS;
constexpr int NB_STAGES = 2;  // 3 leave room for fewer groups: 32768 rows of 5120 bf16 251 us instead of 173
// Groups of threads as in k_norm, each on R rows at a time (2 of bf16, 1 of fp32), so that their exchanges and the
// weights are shared.  One block of 512 threads to an SM, so that a thread has 128 registers for its columns' sums
// (two blocks of half the groups: 184 us instead of 173).
template <typename T, typename P, int NV, bool VEC>
__global__ void __maxnreg__(NB_REGS) k_norm_backward(NormArgs a, int width, bool sums) {
  constexpr int R = sizeof(T) == 4 ? 1 : 2;
  using C = Cols<T, VEC, NV>;
  using S = SharedParams<T, P, VEC, NV>;
  constexpr int PER = C::PER, HALF = PER / 2;
  extern __shared__ __align__(16) unsigned char norm_smem[];
  __shared__ float sh[2][NB_THREADS / 32][2 * R];
  const int group = threadIdx.x / width, groups = blockDim.x / width, me = threadIdx.x - group * width;
  const int warp = threadIdx.x >> 5, lane = me & 31, warps = width >> 5, warp0 = warp - (me >> 5);
  const float inv_d = 1.f / (float)a.d;
  int turn = 0;
  const S w_shared(norm_smem);
  const Ring<T, VEC, NV> ring(norm_smem + S::bytes(width), me, a.d);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (sums) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel follows
  f32x2 dw[NV][HALF], db[NV][HALF];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < HALF; ++e) dw[v][e] = db[v][e] = 0;
  const unsigned rows = a.N, step = gridDim.x * groups * R;
  unsigned n = (blockIdx.x * groups + group) * R;
  const long long x_step = step * a.ld, g_step = step * a.grad_ld, dx_step = step * a.y_ld;
  const T* x_row = static_cast<const T*>(a.x) + n * a.ld;
  const T* g_row = static_cast<const T*>(a.grad) + n * a.grad_ld;
  const T *x_next = x_row + ring.first, *g_next = g_row + ring.first;  // the next rows to fetch
  T* out = a.y ? static_cast<T*>(a.y) + n * a.y_ld : nullptr;
  const float2* st_next = a.stats + n;
  float2 stn[R];
  auto fetch = [&](unsigned first, int s) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      ring.fetch(x_next + i * a.ld, first + i < rows, (s * R + i) * 2);
      ring.fetch(g_next + i * a.grad_ld, first + i < rows, (s * R + i) * 2 + 1);
    }
    x_next += x_step;
    g_next += g_step;
  };
  auto fetch_stats = [&](unsigned first) {
#pragma unroll
    for (int i = 0; i < R; ++i) stn[i] = first + i < rows ? __ldg(st_next + i) : make_float2(0.f, 0.f);
    st_next += step;
  };
#pragma unroll
  for (int s = 0; s < NB_STAGES - 1; ++s) fetch(n + s * step, s);
  fetch_stats(n);
  if (a.weight) w_shared.fill(static_cast<const P*>(a.weight), width, a.d);
  __syncthreads();
  int stage = 0;
  for (; n < rows; n += step) {
    float2 st[R];
#pragma unroll
    for (int i = 0; i < R; ++i) st[i] = stn[i];
    ring.template wait<2 * R * (NB_STAGES - 2)>();
    fetch(n + (NB_STAGES - 1) * step, stage == 0 ? NB_STAGES - 1 : stage - 1);
    fetch_stats(n + step);
    const bool pair = R == 1 || n + 1 < rows;  // the last row may be alone
    // x - mean and g of vector v of row i; past the row's end g is 0 and x - mean counts for nothing
    auto terms = [&](int i, int v, f32x2* z, f32x2* q) {
      const f32x2 shift = both(-st[i].x);
      unpack_pairs<T>(ring.get(x_row + i * a.ld, (stage * R + i) * 2, v), z);
      unpack_pairs<T>(ring.get(g_row + i * a.grad_ld, (stage * R + i) * 2 + 1, v), q);
#pragma unroll
      for (int e = 0; e < HALF; ++e) z[e] = add2(z[e], shift);
    };
    f32x2 s1[R], s2[R];
#pragma unroll
    for (int i = 0; i < R; ++i) s1[i] = s2[i] = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      f32x2 w[HALF];
      if (a.weight) w_shared.pairs(w, me, v);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (i > 0 && !pair) continue;
        f32x2 z[HALF], q[HALF];
        const f32x2 rstd = both(st[i].y);
        terms(i, v, z, q);
#pragma unroll
        for (int e = 0; e < HALF; ++e) {
          dw[v][e] = fma2(q[e], mul2(z[e], rstd), dw[v][e]);
          db[v][e] = add2(db[v][e], q[e]);
          const f32x2 t = a.weight ? mul2(q[e], w[e]) : q[e];
          s1[i] = add2(s1[i], t);
          s2[i] = fma2(t, z[e], s2[i]);
        }
      }
    }
    if (out) {
      // the rows' sums: 2 R values over the block
      float part;
      if constexpr (R == 2) {
        const float p = fold(pair_sum(s1[0]), pair_sum(s1[1]), 16), q = fold(pair_sum(s2[0]), pair_sum(s2[1]), 16);
        part = fold(p, q, 8);
      } else {
        part = fold(pair_sum(s1[0]), pair_sum(s2[0]), 16);
        part += __shfl_xor_sync(0xFFFFFFFFu, part, 8);
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
      // this lane's value: (row, sum) = (lane bit 4, lane bit 3), or for one row the sum = lane bit 4
      constexpr int LANES = R == 2 ? 8 : 16;
      const int which = lane / LANES, k0 = lane % LANES;
      if (warps > 1) {
        if (k0 == 0) sh[turn][warp][which] = part;
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(width) : "memory");
        part = 0.f;
#pragma unroll
        for (int k = 0; k < NB_THREADS / 32; k += LANES)
          if (k0 + k < warps) part += sh[turn][warp0 + k0 + k][which];
        turn ^= 1;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
      }
      // dx = rstd t + (x - mean) c2 + c1
      f32x2 c1[R], c2[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float m1 = -inv_d * __shfl_sync(0xFFFFFFFFu, part, 2 * i * LANES);
        const float m2 = -inv_d * __shfl_sync(0xFFFFFFFFu, part, (2 * i + 1) * LANES);
        c1[i] = both(m1 * st[i].y);
        c2[i] = both(((m2 * st[i].y) * st[i].y) * st[i].y);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        f32x2 w[HALF];
        if (a.weight) w_shared.pairs(w, me, v);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          if (i > 0 && !pair) continue;
          f32x2 z[HALF], t[HALF];
          const f32x2 rstd = both(st[i].y);
          terms(i, v, z, t);
#pragma unroll
          for (int e = 0; e < HALF; ++e) {
            if (a.weight) t[e] = mul2(t[e], w[e]);
            t[e] = fma2(t[e], rstd, fma2(z[e], c2[i], c1[i]));
          }
          C::store(out + i * a.y_ld, me, v, a.d, round_pairs<T>(t));
        }
      }
      out += dx_step;
    }
    x_row += x_step;
    g_row += g_step;
    stage = stage + 1 == NB_STAGES ? 0 : stage + 1;
  }
  if (!sums) return;
  // the block's sums: the groups add theirs one after another, in shared memory, the last one on its way out; in the
  // order of the threads' columns, (v, e) major
  float* part = a.ws + (long long)blockIdx.x * 2 * a.part_ld;
  float* all = reinterpret_cast<float*>(norm_smem);
  ring.template wait<0>();
  for (int k = 0; k < groups; ++k) {
    if (groups > 1) __syncthreads();
    if (group != k) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        float x = half_of(dw[v][e / 2], e & 1), y = half_of(db[v][e / 2], e & 1);
        const int at = (v * PER + e) * width + me, other = NV * PER * width;
        if (k > 0) {
          x += all[at];
          y += all[other + at];
        }
        float* to = k + 1 < groups ? all : part;
        to[at] = x;
        to[(k + 1 < groups ? other : a.part_ld) + at] = y;
      }
    }
  }
}

// ------------------------------------------------------------------ wide rows

constexpr int NW_THREADS = 1024;

template <typename T, typename P>
__global__ void __launch_bounds__(NW_THREADS) k_norm_wide(NormArgs a) {
  __shared__ float2 sh[2][32];
  int turn = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const P* w = static_cast<const P*>(a.weight);
  const P* b = static_cast<const P*>(a.bias);
  const float inv_d = 1.f / (float)a.d;
  for (long long n = blockIdx.x; n < a.N; n += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + n * a.ld;
    T* y = static_cast<T*>(a.y) + n * a.y_ld;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.d; i += NW_THREADS) s += Elem<T>::to_f(x[i]);
    const float mean0 = block_sum(s, 0.f, sh, turn).x * inv_d;
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < a.d; i += NW_THREADS) {
      const float t = Elem<T>::to_f(x[i]) - mean0;
      s1 += t;
      s2 = fmaf(t, t, s2);
    }
    const Moments q = moments(mean0, block_sum(s1, s2, sh, turn), inv_d, a.eps);
    if (a.stats_out && threadIdx.x == 0) a.stats_out[n] = make_float2(q.mean0 + q.delta, q.rstd);
    for (int i = threadIdx.x; i < a.d; i += NW_THREADS) {
      float z = ((Elem<T>::to_f(x[i]) - q.mean0) - q.delta) * q.rstd;
      if (w) z = b ? fmaf(z, Elem<P>::to_f(w[i]), Elem<P>::to_f(b[i])) : z * Elem<P>::to_f(w[i]);
      else if (b) z += Elem<P>::to_f(b[i]);
      y[i] = Elem<T>::from_f(z);
    }
  }
}

template <typename T, typename P>
__global__ void __launch_bounds__(NW_THREADS) k_norm_backward_wide(NormArgs a) {
  __shared__ float2 sh[2][32];
  int turn = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const P* w = static_cast<const P*>(a.weight);
  const float inv_d = 1.f / (float)a.d;
  for (long long n = blockIdx.x; n < a.N; n += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + n * a.ld;
    const T* g = static_cast<const T*>(a.grad) + n * a.grad_ld;
    T* dx = static_cast<T*>(a.y) + n * a.y_ld;
    const float2 st = __ldg(a.stats + n);
    auto terms = [&](int i, float* hat) {
      *hat = (Elem<T>::to_f(x[i]) - st.x) * st.y;
      const float q = Elem<T>::to_f(g[i]);
      return w ? q * Elem<P>::to_f(w[i]) : q;
    };
    float s1 = 0.f, s2 = 0.f, hat;
    for (int i = threadIdx.x; i < a.d; i += NW_THREADS) {
      const float t = terms(i, &hat);
      s1 += t;
      s2 = fmaf(t, hat, s2);
    }
    const float2 c = block_sum(s1, s2, sh, turn);
    const float c1 = c.x * inv_d, c2 = c.y * inv_d;
    for (int i = threadIdx.x; i < a.d; i += NW_THREADS) {
      const float t = terms(i, &hat);
      dx[i] = Elem<T>::from_f(st.y * fmaf(-hat, c2, t - c1));
    }
  }
}

// A sum with what its additions round off (the exact error of a sum, by Knuth).
struct LongSum {
  float sum, rest;
  __device__ __forceinline__ void add(float x) {
    const float s = sum + x, b = s - sum;
    rest += (sum - (s - b)) + (x - b);
    sum = s;
  }
  __device__ __forceinline__ void add(const LongSum& o) {
    add(o.sum);
    rest += o.rest;
  }
  // (an infinite or NaN sum has no remainder)
  __device__ __forceinline__ float value() const { return fabsf(sum) < INFINITY ? sum + rest : sum; }
};

// dw and db of a tile of columns over a share of the rows, NC_RUN of them at a time in one fp32 sum: a share of a
// million rows of 65536 columns is 250000 rows, and their errors would add up.  The runs' sums wait in shared memory
// and four rows are loaded ahead, so that all blocks of the grid run at once with 32 registers (the gradient of
// 10000 rows of 12288 bf16 433 us; 494 with a run unrolled by four, 653 with 40 registers).
constexpr int NC_THREADS = 256, NC_BLOCKS = 8, NC_RUN = 32, NC_AHEAD = 4;
template <typename T>
__global__ void __launch_bounds__(NC_THREADS, NC_BLOCKS) k_norm_columns(NormArgs a) {
  __shared__ LongSum sh[2][NC_THREADS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the kernel that follows may be the gradient's, which may overwrite x or the gradient: it waits for this one to end
  // before it touches memory
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int col = blockIdx.x * NC_THREADS + threadIdx.x;
  if (col >= a.d) return;
  const T* x = static_cast<const T*>(a.x) + col;
  const T* g = static_cast<const T*>(a.grad) + col;
  LongSum& w = sh[0][threadIdx.x];
  LongSum& b = sh[1][threadIdx.x];
  w = b = LongSum{0.f, 0.f};
  const long long x_step = gridDim.y * a.ld, g_step = gridDim.y * a.grad_ld;
  const float2* stats = a.stats + blockIdx.y;
  x += blockIdx.y * a.ld;
  g += blockIdx.y * a.grad_ld;
  int left = (int)((a.N - blockIdx.y + gridDim.y - 1) / gridDim.y);  // (as many blocks as rows at most)
  while (left > 0) {
    float dw = 0.f, db = 0.f;
    auto rows = [&](auto many) {
      constexpr int R = decltype(many)::value;
      float2 st[R];
      float p[R], q[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        st[i] = __ldg(stats);
        p[i] = Elem<T>::to_f(*x);
        q[i] = Elem<T>::to_f(*g);
        stats += gridDim.y;
        x += x_step;
        g += g_step;
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        dw = fmaf(q[i], (p[i] - st[i].x) * st[i].y, dw);
        db += q[i];
      }
    };
    int n = min(left, NC_RUN);
    left -= n;
    for (; n >= NC_AHEAD; n -= NC_AHEAD) rows(std::integral_constant<int, NC_AHEAD>{});
    for (; n > 0; --n) rows(std::integral_constant<int, 1>{});
    w.add(dw);
    b.add(db);
  }
  float* part = a.ws + (long long)blockIdx.y * 2 * a.part_ld;
  part[col] = w.value();
  part[a.part_ld + col] = b.value();
}

// The blocks' sums, added in a fixed order, the last steps without loss, and rounded once.  They stand in the order
// of the threads' columns, nv vectors of `per` of a thread and `width` threads (nv 0: in the order of the columns).
constexpr int NJ_COLS = 32, NJ_ROWS = 32;
template <typename P>
__global__ void __launch_bounds__(NJ_COLS * NJ_ROWS) k_norm_join(NormArgs a, int parts, int width, int nv, int per,
                                                                 bool vec) {
  __shared__ float sh[NJ_ROWS][NJ_COLS + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, at = blockIdx.x * NJ_COLS + lane;
  P* out = static_cast<P*>(blockIdx.y ? a.grad_bias : a.grad_weight);
  if (!out) return;
  const float* from = a.ws + blockIdx.y * a.part_ld + at;
  float s = 0.f;
  if (at < a.part_ld) {
#pragma unroll 8
    for (int i = row; i < parts; i += NJ_ROWS) s += from[(long long)i * 2 * a.part_ld];
  }
  sh[row][lane] = s;
  __syncthreads();
  // warp r adds up column r: lane l has part l's sum
  LongSum t = {sh[lane][row], 0.f};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    LongSum other;
    other.sum = __shfl_xor_sync(0xFFFFFFFFu, t.sum, o);
    other.rest = __shfl_xor_sync(0xFFFFFFFFu, t.rest, o);
    t.add(other);
  }
  if (lane != 0) return;
  const int mine = blockIdx.x * NJ_COLS + row;
  int id = mine;
  if (nv > 0) {
    const int thread = mine % width, ve = mine / width;
    id = (thread >> 5) * (32 * nv * per) +
         (vec ? ((ve / per) * 32 + (thread & 31)) * per + ve % per : ve * 32 + (thread & 31));
  }
  if (id < a.d) out[id] = Elem<P>::from_f(t.value());
}

// Blocks that leave sums, at most: 2^22 columns of them, or 512.
int norm_parts(int d) { return (1 << 22) / d < 512 ? (1 << 22) / d : 512; }

int round32(int x) { return (x + 31) / 32 * 32; }
unsigned least(long long a, long long b) { return (unsigned)(a < b ? a : b); }

// Lets a kernel take as much shared memory as the device has, once per (kernel, device).
cudaError_t allow_ring(const void* kernel, int device) {
  static std::mutex mu;
  static std::vector<std::pair<const void*, int>> done;
  std::lock_guard<std::mutex> lk(mu);
  for (const auto& d : done)
    if (d.first == kernel && d.second == device) return cudaSuccess;
  int most = 0;
  cudaFuncAttributes fa;
  cudaError_t e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)fa.sharedSizeBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return note_error(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
  done.emplace_back(kernel, device);
  return cudaSuccess;
}
// Launches a kernel whose ring takes `smem` bytes of shared memory.
template <class Kernel, class... A>
cudaError_t launch_ring(const Ctx& c, const char* name, Kernel* kernel, unsigned grid, unsigned threads, size_t smem,
                        A... args) {
  const cudaError_t e = smem > 0 ? allow_ring(reinterpret_cast<const void*>(kernel), c.device) : cudaSuccess;
  return e != cudaSuccess ? e : launch_pdl(c, name, kernel, dim3(grid), dim3(threads), smem, args...);
}

constexpr int SM_SMEM = 220 * 1024;  // of an SM's shared memory, for the rings of its blocks

template <typename T, typename P, bool VEC, int NV>
cudaError_t run_norm_nv(const Ctx& c, const NormArgs& a, int nvec, bool few) {
  const int width = round32((nvec + NV - 1) / NV);
  const size_t ring = NF_STAGES * Ring<T, VEC, NV>::bytes(width);
  const size_t shared = 2 * SharedParams<T, P, VEC, NV>::bytes(width);
  const int barriers = width > 32 ? 15 : 32;  // one per group, but for rows of one warp
  auto groups_by = [&](int regs) {
    const long long fit = (SM_SMEM - (long long)shared) / (long long)ring;
    const unsigned groups = least(least(threads_by_regs(regs) / width, barriers), fit);
    return groups < 1 ? 1u : groups;
  };
  auto run = [&](auto kernel, unsigned groups) {
    const unsigned grid = least(((long long)a.N + groups - 1) / groups, c.num_sms);
    return launch_ring(c, "norm", kernel, grid, (unsigned)width * groups, shared + ring * groups, a, width);
  };
  auto pick = [&](auto end) {
    constexpr RowEnd S = decltype(end)::value;
    if (few)
      return launch_ring(c, "norm", k_norm<T, P, NV, VEC, S, false, norm_regs(NV)>, (unsigned)a.N, (unsigned)width,
                         ring, a, width);
    const unsigned groups = groups_by(norm_regs(NV));
    if constexpr (NV == 4)
      if (groups_by(NF_TIGHT) > groups) return run(k_norm<T, P, NV, VEC, S, true, NF_TIGHT>, groups_by(NF_TIGHT));
    return run(k_norm<T, P, NV, VEC, S, true, norm_regs(NV)>, groups);
  };
  const int last = a.d % Cols<T, VEC, NV>::WARP;  // columns of a warp that the row ends in
  if constexpr (NV > 1)
    if (width > 32 && last > 0 && last < 8 * 32) return pick(std::integral_constant<RowEnd, SHORT>{});
  if constexpr (VEC && NV == 4)
    if (last == 0) return pick(std::integral_constant<RowEnd, WHOLE>{});
  return pick(std::integral_constant<RowEnd, LONG>{});
}

template <typename T, typename P, bool VEC>
cudaError_t run_norm(const Ctx& c, const NormArgs& a) {
  constexpr int PER = Elem<T>::PER16;
  const int nvec = (a.d + PER - 1) / PER;
  // one row per block and no parameters in shared memory where there are few rows (5120 bf16: 8 rows 2.6 us, 4.0 as
  // many rows are done; 304 rows 3.3 and 4.1; 608 rows 5.9 and 4.3)
  const bool few = a.N <= 2 * c.num_sms;
  if (nvec <= 32) return run_norm_nv<T, P, VEC, 1>(c, a, nvec, few);
  if (nvec <= 64 || (few && nvec <= 2 * 32 * NF_WARPS)) return run_norm_nv<T, P, VEC, 2>(c, a, nvec, few);
  // (32768 rows of 5120 bf16 with 2 vectors per thread 135 us instead of 103)
  return run_norm_nv<T, P, VEC, 4>(c, a, nvec, few);
}

// How the backward pass left its sums.
struct JoinPlan {
  int parts, width, nv, per;
  bool vec;
};

template <typename T, typename P, bool VEC, int NV>
cudaError_t run_backward_nv(const Ctx& c, NormArgs& a, bool sums, JoinPlan* join, int nvec) {
  constexpr int PER = Elem<T>::PER16, R = sizeof(T) == 4 ? 1 : 2;
  const int width = round32((nvec + NV - 1) / NV);
  const size_t ring = NB_STAGES * 2 * R * Ring<T, VEC, NV>::bytes(width);
  const size_t shared = SharedParams<T, P, VEC, NV>::bytes(width);
  const long long units = ((long long)a.N + R - 1) / R;
  long long groups = NB_THREADS / width;
  if (shared + ring * groups > SM_SMEM) groups = (SM_SMEM - (long long)shared) / (long long)ring;
  groups = least(groups < 1 ? 1 : groups, 15);  // a barrier each
  // few rows: on as many SMs as there are
  if (units < c.num_sms * groups) groups = (units + c.num_sms - 1) / c.num_sms;
  size_t smem = shared + ring * groups;
  const size_t joined = (size_t)width * NV * PER * 2 * sizeof(float);  // the groups' sums
  if (groups > 1 && joined > smem) smem = joined;
  *join = {(int)least((units + groups - 1) / groups, least(norm_parts(a.d), c.num_sms)), width, NV, PER, VEC};
  a.part_ld = width * NV * PER;
  return launch_ring(c, "norm_backward", k_norm_backward<T, P, NV, VEC>, (unsigned)join->parts,
                     (unsigned)(width * groups), smem, a, width, sums);
}

template <typename T, typename P, bool VEC>
cudaError_t run_norm_backward(const Ctx& c, NormArgs& a, bool sums, JoinPlan* join) {
  const int nvec = (a.d + Elem<T>::PER16 - 1) / Elem<T>::PER16;
  if constexpr (sizeof(T) == 4) {
    if (nvec <= 512) return run_backward_nv<T, P, VEC, 2>(c, a, sums, join, nvec);
    return run_backward_nv<T, P, VEC, 4>(c, a, sums, join, nvec);
  } else {
    // two vectors per thread, or three where whole groups of two would leave more than a fifth of the threads out
    // (32768 rows of 5120: 189 us with two, 173 with three; of 1024: 39 and 53; of 2048: 65 and 76)
    const int two = round32((nvec + 1) / 2), three = round32((nvec + 2) / 3);
    if (NB_THREADS / two * two * 5 / 4 >= NB_THREADS / three * three)
      return run_backward_nv<T, P, VEC, 2>(c, a, sums, join, nvec);
    return run_backward_nv<T, P, VEC, 3>(c, a, sums, join, nvec);
  }
}

bool params16(const void* w, const void* b) {
  return ((reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(b)) & 15u) == 0;
}

template <typename T, typename P>
cudaError_t pick_norm(const Ctx& c, const NormArgs& a) {
  if (a.d > NM_HELD)
    return launch_pdl(c, "norm", k_norm_wide<T, P>, dim3(least(a.N, 2LL * c.num_sms)), dim3(NW_THREADS), 0, a);
  const bool vec = params16(a.weight, a.bias) && whole_vectors(a.x, a.ld, a.N, a.d, sizeof(T)) &&
                   whole_vectors(a.y, a.y_ld, a.N, a.d, sizeof(T));
  return vec ? run_norm<T, P, true>(c, a) : run_norm<T, P, false>(c, a);
}

template <typename T, typename P>
cudaError_t pick_backward(const Ctx& c, NormArgs a) {
  const bool sums = a.grad_weight || a.grad_bias;
  JoinPlan join = {};
  a.part_ld = a.d;
  cudaError_t e = cudaSuccess;
  if (a.N == 0) {
    // sums of no rows: the joining kernel writes zeros
  } else if (a.d <= NM_HELD) {
    const bool vec = params16(a.weight, nullptr) && whole_vectors(a.x, a.ld, a.N, a.d, sizeof(T)) &&
                     whole_vectors(a.grad, a.grad_ld, a.N, a.d, sizeof(T)) &&
                     (!a.y || whole_vectors(a.y, a.y_ld, a.N, a.d, sizeof(T)));
    e = vec ? run_norm_backward<T, P, true>(c, a, sums, &join) : run_norm_backward<T, P, false>(c, a, sums, &join);
  } else {
    // the columns' sums first: the gradient may overwrite the rows
    if (sums) {
      const int tiles = (a.d + NC_THREADS - 1) / NC_THREADS, shares = NC_BLOCKS * c.num_sms / tiles;
      join.parts = (int)least(a.N, least(norm_parts(a.d), shares < 1 ? 1 : shares));
      e = launch_pdl(c, "norm_columns", k_norm_columns<T>, dim3((unsigned)tiles, (unsigned)join.parts),
                     dim3(NC_THREADS), 0, a);
    }
    if (e == cudaSuccess && a.y)
      e = launch_pdl(c, "norm_backward", k_norm_backward_wide<T, P>, dim3(least(a.N, 2LL * c.num_sms)),
                     dim3(NW_THREADS), 0, a);
  }
  if (e != cudaSuccess || !sums) return e;
  return launch_pdl(c, "norm_join", k_norm_join<P>, dim3((unsigned)((a.part_ld + NJ_COLS - 1) / NJ_COLS), 2u),
                    dim3(NJ_COLS * NJ_ROWS), 0, a, join.parts, join.width, join.nv, join.per, join.vec);
}

}  // namespace

// (a block's threads have up to 1024 columns more than the row)
size_t norm_backward_workspace(int N, int d, int) {
  return WS_HEADER + align_up((size_t)least(N, norm_parts(d)) * 2 * (d + 1024) * sizeof(float), 256);
}

cudaError_t launch_norm(const Ctx& c, const NormArgs& a, int dtype, int param_dtype) {
  if (dtype == DH_F32) return pick_norm<float, float>(c, a);
  return param_dtype == DH_F32 ? pick_norm<__nv_bfloat16, float>(c, a)
                               : pick_norm<__nv_bfloat16, __nv_bfloat16>(c, a);
}
cudaError_t launch_norm_backward(const Ctx& c, const NormArgs& a, int dtype, int param_dtype) {
  if (dtype == DH_F32) return pick_backward<float, float>(c, a);
  return param_dtype == DH_F32 ? pick_backward<__nv_bfloat16, float>(c, a)
                               : pick_backward<__nv_bfloat16, __nv_bfloat16>(c, a);
}

}  // namespace dh
