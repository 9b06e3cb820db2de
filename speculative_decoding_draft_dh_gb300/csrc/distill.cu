// Distillation from a teacher's top logits: the loss of a student's rows of logits and its gradient
// (definitions at dh_distill_topk in dh.h).
//
// With p = softmax(y / T) over the teacher's entries and q = softmax(z / T) over the vocabulary,
//   loss = T^2 sum_k p_k (log p_k - log q[id_k]),   dz[v] = g T (q[v] - sum of the p_k with id_k = v).
// Only the normaliser of q needs the whole row; the entries are a sparse correction of the dense
// term g T q.  So every form is a statistics pass, a dense pass (both bound by HBM) and a small
// kernel for the entries:
//   loss              k_row_stats (row_stats.cu), k_distill_finish
//   gradient          k_distill_dense, k_distill_finish
//   both              k_distill_ring (distill_ring.cu: statistics and dense term in one pass over the
//                     logits), k_distill_finish
//   gradient where the rows do not lie like their logits, or in the logits' place: k_distill_grad
//   short rows: k_distill_short, one block per row, everything in one launch
//
// k_distill_dense: the exponentials of a row's vectors times one factor; `splits` blocks per row.
//   1024 rows of 151936 bf16 logits, 622 MB: 91 us, 6.4 TB/s with the rows that are not read taken
//   off.  Eight vectors per thread of 512 in flight; measured against 4 per thread of 256: 98 us.
// k_distill_finish: one warp per row: the teacher's softmax, the loss, and the entries' values over
//   the dense ones, one writer per id: the first entry of an id adds up the others' p in order, so
//   repeated ids repeat bit for bit.  A hash table in shared memory finds out whether there are any.
//   Latency-bound (ids, then their logits, then the row's statistics), so it starts under the pass
//   before it by programmatic dependent launch and waits for that pass only when it needs the
//   statistics (2048 rows of 64 entries: 12 us after a pass, 7 where it can start under it).  What it
//   reads before the wait are the call's inputs: the kernels before it let it start only after their
//   own wait, when those are complete.
// k_distill_grad: dense term and entries in one kernel; the logits of a part's entries are read
//   before its dense pass writes anything.

#include "rows.cuh"

namespace dh {
namespace {

constexpr int DF_WARPS = 4;
constexpr int DS_WARPS = 8;
// Rows for one block and one launch.  Measured in graphs, us, bf16, this against two launches: loss of
// 16 x 8192 5.7 / 6.8, of 608 x 16384 (16 segments) 10.5 / 10.8, of 2048 x 8192 15.2 / 13.5; gradient
// of 608 x 16384 16.5 / 17.2, of 2048 x 16384 35.0 / 30.7; step of 16 x 8192 9.0 / 10.8, of 608 x 32768
// (32 segments) 23.5 / 31.0, of 16 x 32768 12.4 / 11.5, of 2048 x 65536 (64 segments) 123 / 106.
constexpr int DS_SEG_FEW = 16;
constexpr int DS_MAX_SEG = 32;
constexpr int DF_BATCH = 8;
constexpr int DG_THREADS = 256;
constexpr int DG_UNROLL = 4;
constexpr int DD_THREADS = 512;
constexpr int DD_UNROLL = 8;

template <int NT>
__device__ __forceinline__ float block_max(float x, float* red) {
  x = warp_max(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float m = red[0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) m = max_nan(m, red[w]);
  return m;
}
template <int NT>
__device__ __forceinline__ float block_sum(float x, float* red) {
  x = warp_sum(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) s += red[w];
  return s;
}

// The teacher's entries of one row: s_id[k] (-1: not an entry) and s_p[k], k < nk.
struct Teacher {
  float top, log_total;  // log p_k = (y_k - top) / T - log_total
  bool any;              // there is an entry above -inf (or a NaN one)
};

template <int NT>
__device__ __forceinline__ Teacher teacher_row(const int32_t* __restrict__ idx, const float* __restrict__ y, int nk,
                                               int vocab, float inv_t, int32_t* s_id, float* s_p, float* red) {
  Teacher t;
  float top = -INFINITY;
  for (int k = threadIdx.x; k < nk; k += NT) {
    const int32_t id = __ldg(idx + k);
    const bool in = id >= 0 && id < vocab;
    const float v = in ? __ldg(y + k) : -INFINITY;
    s_id[k] = in ? id : -1;
    s_p[k] = v;
    top = max_nan(top, v);
  }
  t.top = block_max<NT>(top, red);
  t.any = t.top != -INFINITY;
  t.log_total = 0.f;
  if (!t.any) return t;
  float sum = 0.f;
  for (int k = threadIdx.x; k < nk; k += NT) {
    const float e = expf((s_p[k] - t.top) * inv_t);
    s_p[k] = e;
    sum += e;
  }
  const float total = block_sum<NT>(sum, red);
  const float inv = 1.f / total;
  t.log_total = logf(total);
  for (int k = threadIdx.x; k < nk; k += NT) s_p[k] *= inv;
  return t;
}

// Loads that may see memory which this kernel writes later (the gradient in the logits' place).
__device__ __forceinline__ uint4 ld16_rw(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ void st16(void* p, const uint4& v) {
  asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// One vector of a row that does not start on the 16 bytes that the output does: element by element.
template <typename T>
__device__ __forceinline__ uint4 ld16_elems(const T* p) {
  constexpr int PER = Elem<T>::PER16;
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    if constexpr (sizeof(T) == 4) w[e] = elem_bits(*(const volatile float*)(p + e));
    else w[e / 2] |= (uint32_t)(*(const volatile unsigned short*)(p + e)) << (16 * (e & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__global__ void __launch_bounds__(DG_THREADS) k_distill_grad(DistillArgs a) {
  constexpr int PER = Elem<T>::PER16;
  __shared__ int32_t s_id[DH_MAX_K];
  __shared__ float s_p[DH_MAX_K];
  __shared__ float s_z[DH_MAX_K];
  __shared__ float red[DG_THREADS / 32];
  const int row = blockIdx.x / a.splits, part = blockIdx.x - row * a.splits;
  const int32_t* idx = a.idx + (size_t)row * a.K;
  const float* y = a.teacher + (size_t)row * a.K;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const T* z = static_cast<const T*>(a.logits) + (size_t)row * a.ld;
  T* out = static_cast<T*>(a.grad) + (size_t)row * a.gld;
  const int nk = a.n_valid ? min(max(__ldg(a.n_valid + row), 0), a.K) : a.K;
  const float g = __ldg(a.weight + row) * a.temperature;
  const int tid = threadIdx.x;

  // the block's part of the row on the output's 16-byte grid: [lo, hi), vectors from vlo to vhi
  // counted from element `pre`; the first part takes the elements before, the last those behind
  const int pre = min(a.vocab, (int)(((16u - (unsigned)(reinterpret_cast<uintptr_t>(out) & 15u)) & 15u) / sizeof(T)));
  const int nvec = (a.vocab - pre) / PER;
  const int vlo = (int)((long long)nvec * part / a.splits), vhi = (int)((long long)nvec * (part + 1) / a.splits);
  const int lo = part == 0 ? 0 : pre + vlo * PER, hi = part == a.splits - 1 ? a.vocab : pre + vhi * PER;

  const float2 st = __ldg(a.stats + row);
  const float m = st.x, sum = st.y;
  const Teacher t = teacher_row<DG_THREADS>(idx, y, nk, a.vocab, a.inv_t, s_id, s_p, red);
  if (!t.any || g == 0.f) {  // nothing to learn from this row: zeros, and its logits are not read
    for (int i = lo + tid; i < min(hi, pre); i += DG_THREADS) out[i] = Elem<T>::from_f(0.f);
    for (int j = vlo + tid; j < vhi; j += DG_THREADS) st16(out + pre + (long long)j * PER, make_uint4(0, 0, 0, 0));
    for (int i = max(lo, pre + vhi * PER) + tid; i < hi; i += DG_THREADS) out[i] = Elem<T>::from_f(0.f);
    return;
  }
  for (int k = tid; k < nk; k += DG_THREADS) {
    const int id = s_id[k];
    if (id >= lo && id < hi) s_z[k] = Elem<T>::to_f(z[id]);
  }
  __syncthreads();  // every entry's logit is held before the pass below may overwrite it

  // a row of -inf has q = 0 everywhere
  const bool nothing = m == -INFINITY;
  // a NaN among the teacher's entries (its total then is one) makes the whole row NaN
  const ExpRef ref(nothing ? 0.f : m, a.c);
  const float aq = t.log_total != t.log_total ? t.log_total : (nothing ? 0.f : ref.by_max(g / sum, a.c));
  const T* zv = z + pre;
  const bool same = ((reinterpret_cast<uintptr_t>(zv)) & 15u) == 0;
  auto scalar = [&](int i) { out[i] = Elem<T>::from_f(aq * one_exp(Elem<T>::to_f(z[i]), ref, a.c)); };
  if (part == 0)
    for (int i = tid; i < pre; i += DG_THREADS) scalar(i);
  if (part == a.splits - 1)
    for (int i = pre + nvec * PER + tid; i < a.vocab; i += DG_THREADS) scalar(i);
  for (int j = vlo + tid; j < vhi; j += DG_THREADS * DG_UNROLL) {
    uint4 u[DG_UNROLL];
#pragma unroll
    for (int q = 0; q < DG_UNROLL; ++q) {
      const int jj = j + q * DG_THREADS;
      if (jj < vhi) u[q] = same ? ld16_rw(zv + (long long)jj * PER) : ld16_elems<T>(zv + (long long)jj * PER);
    }
#pragma unroll
    for (int q = 0; q < DG_UNROLL; ++q) {
      const int jj = j + q * DG_THREADS;
      if (jj < vhi) st16(out + pre + (long long)jj * PER, grad_vec<T>(u[q], ref, a.c, aq));
    }
  }
  __syncthreads();  // the entries' values below come after the dense ones
  for (int k = tid; k < nk; k += DG_THREADS) {
    const int id = s_id[k];
    if (id < lo || id >= hi) continue;
    float p = s_p[k];
    bool first = true;
    for (int j = 0; j < nk; ++j) {
      if (s_id[j] != id || j == k) continue;
      if (j < k) { first = false; break; }
      p += s_p[j];
    }
    if (first) out[id] = Elem<T>::from_f(aq * one_exp(s_z[k], ref, a.c) - g * p);
  }
}

// ---------------------------------------------------------------- dense term

template <typename T>
__global__ void __launch_bounds__(DD_THREADS) k_distill_dense(DistillArgs a) {
  constexpr int PER = Elem<T>::PER16;
  const int row = blockIdx.x / a.splits, part = blockIdx.x - row * a.splits;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // only now: k_distill_finish reads the call's inputs as soon as it may start
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const T* z = static_cast<const T*>(a.logits) + (long long)row * a.ld;
  T* out = static_cast<T*>(a.grad) + (long long)row * a.gld;
  const int tid = threadIdx.x;
  const int pre = min(a.vocab, (int)(((16u - (unsigned)(reinterpret_cast<uintptr_t>(z) & 15u)) & 15u) / sizeof(T)));
  const int nvec = (a.vocab - pre) / PER;
  const int vlo = (int)((long long)nvec * part / a.splits), vhi = (int)((long long)nvec * (part + 1) / a.splits);
  const float2 st = __ldg(a.stats + row);
  const float g = __ldg(a.weight + row) * a.temperature;
  const bool zero = g == 0.f || (a.n_valid && __ldg(a.n_valid + row) <= 0);
  const bool nothing = st.x == -INFINITY;  // a row of -inf has q = 0 everywhere
  const ExpRef ref(nothing ? 0.f : st.x, a.c);
  const float aq = nothing ? 0.f : ref.by_max(g / st.y, a.c);
  const T* zv = z + pre;
  T* ov = out + pre;
  if (part == 0) {
    const int behind = pre + nvec * PER;
    const int i = tid < pre ? tid : behind + tid - pre;
    if (i < a.vocab) out[i] = Elem<T>::from_f(zero ? 0.f : aq * one_exp(Elem<T>::to_f(z[i]), ref, a.c));
  }
  if (zero) {
    for (int j = vlo + tid; j < vhi; j += DD_THREADS) st16(ov + (long long)j * PER, make_uint4(0, 0, 0, 0));
    return;
  }
  for (int j = vlo + tid; j < vhi; j += DD_THREADS * DD_UNROLL) {
    uint4 u[DD_UNROLL];
#pragma unroll
    for (int q = 0; q < DD_UNROLL; ++q)
      if (j + q * DD_THREADS < vhi) u[q] = ld_nc_v4(zv + (long long)(j + q * DD_THREADS) * PER);
#pragma unroll
    for (int q = 0; q < DD_UNROLL; ++q)
      if (j + q * DD_THREADS < vhi)
        st16(ov + (long long)(j + q * DD_THREADS) * PER, grad_vec<T>(u[q], ref, a.c, aq));
  }
}

// ---------------------------------------------------------------- entries

// The logits of all entries (0 where there is none), for a gradient that overwrites them.
template <typename T>
__global__ void __launch_bounds__(256) k_distill_gather(DistillArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)a.N * a.K) return;
  const int id = __ldg(a.idx + i);
  const long long row = i / a.K;
  a.gathered[i] =
      id >= 0 && id < a.vocab ? Elem<T>::to_f(static_cast<const T*>(a.logits)[row * a.ld + id]) : 0.f;
}

// What one warp knows of a row's entries before it has the row's statistics.
struct RowEntries {
  int nk;
  bool any;      // there is an entry above -inf (or a NaN one)
  bool twice;    // an id comes more than once
  float g;       // grad_loss T
  float total;   // NaN if an entry is
  float part;    // sum_k p_k ((y_k - top)/T - (z_k - zref)/T)
  float pa, pz;  // where that has no finite value: sum_k p_k (y_k - top)/T and sum_k p_k (zref - z_k)/4
  float zref;    // one of the entries' logits
};

// Shared memory of a warp: the entries' ids, p and logits [K], then a hash table (a power of two of
// at least 2 K; only for a gradient).
struct EntrySmem {
  int32_t* id;
  float *p, *z;
  int32_t* table;
  int size;
  __device__ EntrySmem(int32_t* base, int K, int size_) : id(base), size(size_) {
    p = reinterpret_cast<float*>(base + K);
    z = p + K;
    table = base + 3 * K;
  }
};

// By one warp: the teacher's softmax and its part of the loss.  Reads nothing but the call's inputs.
template <typename T, bool LOSS, bool GRAD>
__device__ __forceinline__ RowEntries entries_prepare(const DistillArgs& a, int row, const EntrySmem& s) {
  const int lane = threadIdx.x & 31;
  const T* const z = static_cast<const T*>(a.logits) + (long long)row * a.ld;
  const long long e0 = (long long)row * a.K;
  RowEntries r;
  if (GRAD)
    for (int i = lane; i < s.size; i += 32) s.table[i] = -1;
  const int nk = r.nk = a.n_valid ? min(max(__ldg(a.n_valid + row), 0), a.K) : a.K;
  r.g = GRAD ? __ldg(a.weight + row) * a.temperature : 0.f;
  // DF_BATCH entries per lane at a time: their loads, which hang on nothing, are in flight together
  float top = -INFINITY, zref = -INFINITY;
  for (int k0 = lane; k0 < a.K; k0 += 32 * DF_BATCH) {
    int id[DF_BATCH];
    float y[DF_BATCH], zk[DF_BATCH];
#pragma unroll
    for (int e = 0; e < DF_BATCH; ++e) {
      const int k = k0 + e * 32;
      id[e] = k < a.K ? __ldg(a.idx + e0 + k) : -1;
      y[e] = k < a.K ? __ldg(a.teacher + e0 + k) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < DF_BATCH; ++e) {
      const int k = k0 + e * 32;
      if (k >= nk || id[e] < 0 || id[e] >= a.vocab) id[e] = -1;
      zk[e] = 0.f;
      if (id[e] >= 0)
        zk[e] = a.gathered ? __ldcg(a.gathered + e0 + k) : Elem<T>::to_f(*(const volatile T*)(z + id[e]));
    }
#pragma unroll
    for (int e = 0; e < DF_BATCH; ++e) {
      const int k = k0 + e * 32;
      if (k >= nk) continue;
      if (id[e] < 0) y[e] = -INFINITY;
      else zref = max_nan(zref, zk[e]);
      s.id[k] = id[e];
      s.p[k] = y[e];
      s.z[k] = zk[e];
      top = max_nan(top, y[e]);
    }
  }
  top = warp_max(top);
  zref = warp_max(zref);
  r.zref = fabsf(zref) < INFINITY ? zref : 0.f;
  r.any = top != -INFINITY;
  float total = 0.f;
  if (r.any)
    for (int k = lane; k < nk; k += 32) {
      const float e = expf((s.p[k] - top) * a.inv_t);
      total += e;
    }
  total = r.total = warp_sum(total);
  const float inv = 1.f / total;
  const bool write = GRAD && r.any && r.g != 0.f;
  __syncwarp();  // the table is cleared before any lane looks into it (shuffles order no memory)
  float part = 0.f;
  bool twice = false;
  for (int k = lane; r.any && k < nk; k += 32) {
    const int id = s.id[k];
    const float ak = (s.p[k] - top) * a.inv_t, p = expf(ak) * inv;
    s.p[k] = p;
    if (id < 0) continue;
    if (LOSS && p != 0.f) part += p * (ak - (s.z[k] - r.zref) * a.inv_t);  // 0 log 0 = 0
    if (write) {
      // multiplicative hashing: the product's leading bits; the table is at most half full, so it ends
      for (uint32_t h = (uint32_t)id * 0x9E3779B1u >> (__clz(s.size) + 1);; ++h) {
        const int old = atomicCAS(&s.table[h & (uint32_t)(s.size - 1)], -1, id);
        if (old == -1) break;
        if (old == id) {
          twice = true;
          break;
        }
      }
    }
  }
  r.part = r.pa = LOSS ? warp_sum(part) : 0.f;
  r.pz = 0.f;
  if (LOSS && !(fabsf(r.part) < INFINITY)) {
    // -inf at an entry, or a logit near the type's lowest value, whose quotient by T overflows: the two
    // sums apart, the logits' before it is divided (a quarter of it: the shares may add up to more than 1).
    // A share below fp32's normal numbers counts there, so it is taken as a square of exp(a / 2)
    float pa = 0.f, pz = 0.f;
    for (int k = lane; k < nk; k += 32) {
      const float p = s.p[k];
      if (s.id[k] < 0 || p == 0.f) continue;
      const float ak = (__ldg(a.teacher + e0 + k) - top) * a.inv_t, half = expf(0.5f * ak);
      pa += p * ak;
      pz += half * inv * (half * (0.25f * r.zref - 0.25f * s.z[k]));
    }
    r.pa = warp_sum(pa);
    r.pz = warp_sum(pz);
  }
  r.twice = __any_sync(0xFFFFFFFFu, twice);
  __syncwarp();  // entries_write reads the other lanes' ids and p
  return r;
}

// The row's loss: sum_k p_k (log p_k - log q_k) with log p_k = (y_k - top)/T - log total and
// log q_k = (z_k - m)/T - log sum; for a row of -inf infinite.  The logarithms of the two sums are
// several times the loss and nearly cancel, so they are added in two floats.
__device__ __forceinline__ float entries_loss(const DistillArgs& a, const RowEntries& r, float m, float sum) {
  if (!r.any) return 0.f;
  if (r.total != r.total) return r.total;
  if (m == -INFINITY) return INFINITY;
  if (!(fabsf(m) < INFINITY) || !(sum < INFINITY)) return NAN;  // a NaN or +inf in the row
  const float x = (m - r.zref) * a.inv_t;
  Sum2 l = log_sum(sum, 0.f);
  const Sum2 t = log_sum(r.total, 0.f);
  if (!(fabsf(r.part + x) < INFINITY))  // infinite where an entry's q is 0
    return a.temperature * a.temperature * (r.pa + ((l.hi - t.hi) + (l.lo - t.lo))) +
           4.f * a.temperature * (r.pz + (0.25f * m - 0.25f * r.zref));
  l.add(-t.hi);
  l.add(x);
  l.add(r.part);
  return a.temperature * a.temperature * (l.hi + (l.lo - t.lo));
}

// By the same warp: the entries' values over the dense term.
template <typename T>
__device__ __forceinline__ void entries_write(const DistillArgs& a, T* out, const RowEntries& r, const EntrySmem& s,
                                              float m, float sum) {
  const bool nothing = m == -INFINITY;
  const ExpRef ref(nothing ? 0.f : m, a.c);
  const float aq = nothing ? 0.f : ref.by_max(r.g / sum, a.c);
  for (int k = threadIdx.x & 31; k < r.nk; k += 32) {
    const int id = s.id[k];
    if (id < 0) continue;
    float p = s.p[k];
    bool first = true;
    if (r.twice)
      for (int j = 0; j < r.nk; ++j) {
        if (s.id[j] != id || j == k) continue;
        if (j < k) {
          first = false;
          break;
        }
        p += s.p[j];
      }
    if (first) out[id] = Elem<T>::from_f(aq * one_exp(s.z[k], ref, a.c) - r.g * p);
  }
}

// LOSS: write the loss (and stats_out).  GRAD: write the entries' gradient.  SEG: the row's statistics
// come as its segments' pairs.
template <typename T, bool LOSS, bool GRAD, bool SEG>
__global__ void __launch_bounds__(DF_WARPS * 32) k_distill_finish(DistillArgs a, int table) {
  extern __shared__ int32_t df_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * DF_WARPS + warp;
  const EntrySmem s(df_smem + warp * (3 * a.K + table), a.K, table);
  if (!GRAD) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const RowEntries r = entries_prepare<T, LOSS, GRAD>(a, row < a.N ? row : a.N - 1, s);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= a.N) return;
  float m, sum;
  if (SEG) {
    Sum2 t;
    row_combine(a.seg + (long long)row * a.n_seg, a.n_seg, a.inv_t, &m, &t);
    sum = t.hi + t.lo;
    if (a.stats_out && lane == 0) a.stats_out[row] = make_float2(m, sum);
  } else {
    const float2 st = __ldcg(a.stats + row);
    m = st.x;
    sum = st.y;
  }
  if (LOSS && lane == 0) a.loss_out[row] = entries_loss(a, r, m, sum);
  if (!GRAD || r.g == 0.f) return;
  T* const out = static_cast<T*>(a.grad) + (long long)row * a.gld;
  if (r.any && r.total == r.total) {
    entries_write<T>(a, out, r, s, m, sum);
  } else if (r.nk > 0) {
    // the dense pass knows a row without entries by its count alone, and no NaN among the entries
    for (int i = lane; i < a.vocab; i += 32) out[i] = Elem<T>::from_f(r.any ? r.total : 0.f);
  }
}

// ---------------------------------------------------------------- short rows

// A whole row by one block: DS_WARPS warps take its segments, one more its entries; then all of them
// the dense term.  One launch instead of two.  STATS: the statistics are given.
template <typename T, bool LOSS, bool GRAD, bool STATS>
__global__ void __launch_bounds__(DS_WARPS * 32 + 32) k_distill_short(DistillArgs a, int table) {
  constexpr int PER = Elem<T>::PER16;
  constexpr int NT = DS_WARPS * 32 + 32;
  extern __shared__ int32_t df_smem[];
  __shared__ float2 s_seg[DS_MAX_SEG];
  __shared__ float s_any;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.x;
  const EntrySmem s(df_smem, a.K, table);
  if (!GRAD) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const T* const z = static_cast<const T*>(a.logits) + (long long)row * a.ld;
  RowEntries r = {};
  if (warp == DS_WARPS) {
    r = entries_prepare<T, LOSS, GRAD>(a, row, s);
    if (lane == 0) s_any = !r.any ? 0.f : (r.total == r.total ? 1.f : r.total);
  } else if (!STATS) {
    for (int i = warp; i < a.n_seg; i += DS_WARPS) {
      uint4 u[ROW_SEG_VECS];
      const int id0 = i * row_seg<T>() + lane * PER;
#pragma unroll
      for (int v = 0; v < ROW_SEG_VECS; ++v) u[v] = row_vec_rw<T>(z, id0 + v * 32 * PER, a.vocab);
      const float2 p = segment_stats<T>(u, a.c);
      if (lane == 0) s_seg[i] = p;
    }
  }
  __syncthreads();
  float m, sum;
  if (STATS) {
    const float2 st = __ldg(a.stats + row);
    m = st.x;
    sum = st.y;
  } else {
    Sum2 t;
    row_combine(s_seg, a.n_seg, a.inv_t, &m, &t);
    sum = t.hi + t.lo;
  }
  if (warp == DS_WARPS && lane == 0) {
    if (LOSS) a.loss_out[row] = entries_loss(a, r, m, sum);
    if (!STATS && a.stats_out) a.stats_out[row] = make_float2(m, sum);
  }
  if (!GRAD) return;

  T* const out = static_cast<T*>(a.grad) + (long long)row * a.gld;
  const float g = __ldg(a.weight + row) * a.temperature, any = s_any;
  const bool zero = any == 0.f || g == 0.f, nothing = m == -INFINITY;
  const ExpRef ref(nothing ? 0.f : m, a.c);
  // a NaN among the entries makes the whole row NaN; a row of -inf has q = 0
  const float aq = any != any ? any : (nothing ? 0.f : ref.by_max(g / sum, a.c));
  // vectors on the output's 16-byte grid and the elements beside it
  const int pre = min(a.vocab, (int)(((16u - (unsigned)(reinterpret_cast<uintptr_t>(out) & 15u)) & 15u) / sizeof(T)));
  const int nvec = (a.vocab - pre) / PER, behind = pre + nvec * PER;
  const T* zv = z + pre;
  const bool same = (reinterpret_cast<uintptr_t>(zv) & 15u) == 0;
  const int lone = tid < pre ? tid : behind + tid - pre;
  if (lone < a.vocab)
    out[lone] = Elem<T>::from_f(zero ? 0.f : aq * one_exp(Elem<T>::to_f(*(const volatile T*)(z + lone)), ref, a.c));
  for (int j = tid; j < nvec; j += NT * 2) {
    uint4 u[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (j + q * NT < nvec && !zero)
        u[q] = same ? ld16_rw(zv + (j + q * NT) * PER) : ld16_elems<T>(zv + (j + q * NT) * PER);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (j + q * NT < nvec)
        st16(out + pre + (j + q * NT) * PER, zero ? make_uint4(0, 0, 0, 0) : grad_vec<T>(u[q], ref, a.c, aq));
  }
  __syncthreads();  // the entries' values come after the dense ones
  if (warp == DS_WARPS && !zero && any == any) entries_write<T>(a, out, r, s, m, sum);
}

cudaLaunchConfig_t pdl_config(const Ctx& c, unsigned grid, unsigned block, cudaLaunchAttribute* at) {
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = c.stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T>
cudaError_t run_grad(const Ctx& c, DistillArgs a) {
  // Blocks enough to fill the SMs eight times over, none with less than 2048 vectors.
  const long long vecs = (a.vocab + Elem<T>::PER16 - 1) / Elem<T>::PER16;
  long long splits = (8LL * c.num_sms + a.N - 1) / a.N;
  splits = splits < vecs / 2048 ? splits : vecs / 2048;
  a.splits = (int)(splits > 1 ? splits : 1);
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(c, (unsigned)((long long)a.N * a.splits), DG_THREADS, &at);
  prof_before("distill_grad", c.stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_distill_grad<T>, a);
  prof_after(c.stream);
  return e;
}

template <typename T>
cudaError_t run_dense(const Ctx& c, DistillArgs a) {
  const long long vecs = (a.vocab + Elem<T>::PER16 - 1) / Elem<T>::PER16;
  long long splits = (8LL * c.num_sms + a.N - 1) / a.N;
  splits = splits < vecs / 1024 ? splits : vecs / 1024;
  a.splits = (int)(splits > 1 ? splits : 1);
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(c, (unsigned)((long long)a.N * a.splits), DD_THREADS, &at);
  prof_before("distill_dense", c.stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_distill_dense<T>, a);
  prof_after(c.stream);
  return e;
}

template <typename T>
cudaError_t run_finish(const Ctx& c, const DistillArgs& a, bool loss, bool grad) {
  int table = 0;
  if (grad)
    for (table = 32; table < 2 * a.K;) table *= 2;
  cudaLaunchAttribute at;
  cudaLaunchConfig_t cfg = pdl_config(c, (unsigned)((a.N + DF_WARPS - 1) / DF_WARPS), DF_WARPS * 32, &at);
  cfg.dynamicSmemBytes = (size_t)DF_WARPS * (3 * a.K + table) * 4;  // 80 KB at most
  auto go = [&](auto* kernel, unsigned long long* done) {
    cudaError_t e = cfg.dynamicSmemBytes > 48 * 1024 ? allow_max_smem(kernel, c.device, done) : cudaSuccess;
    // under the ring kernel it needs that kernel's carveout to start; under the others theirs, the
    // default (a changed carveout waits for empty SMs: 68 against 45 us for a loss of 512 rows)
    if (e == cudaSuccess && loss && grad) e = carveout_max_shared((const void*)kernel, c.device);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, a, table);
    return e;
  };
  static unsigned long long done[3] = {};
  prof_before("distill_finish", c.stream);
  cudaError_t e;
  if (loss && grad) e = go(k_distill_finish<T, true, true, false>, &done[0]);
  else if (grad) e = go(k_distill_finish<T, false, true, false>, &done[1]);
  else e = go(k_distill_finish<T, true, false, true>, &done[2]);
  prof_after(c.stream);
  return e;
}

template <typename T>
cudaError_t run_short(const Ctx& c, const DistillArgs& a, bool loss, bool grad) {
  int table = 0;
  if (grad)
    for (table = 32; table < 2 * a.K;) table *= 2;
  cudaLaunchAttribute at;
  cudaLaunchConfig_t cfg = pdl_config(c, (unsigned)a.N, DS_WARPS * 32 + 32, &at);
  cfg.dynamicSmemBytes = (size_t)(3 * a.K + table) * 4;  // 20 KB at most
  prof_before("distill_short", c.stream);
  const cudaError_t e = loss && grad ? cudaLaunchKernelEx(&cfg, k_distill_short<T, true, true, false>, a, table)
                        : grad       ? cudaLaunchKernelEx(&cfg, k_distill_short<T, false, true, true>, a, table)
                                     : cudaLaunchKernelEx(&cfg, k_distill_short<T, true, false, false>, a, table);
  prof_after(c.stream);
  return e;
}

template <typename T>
cudaError_t run_gather(const Ctx& c, const DistillArgs& a) {
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(c, (unsigned)(((long long)a.N * a.K + 255) / 256), 256, &at);
  prof_before("distill_gather", c.stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_distill_gather<T>, a);
  prof_after(c.stream);
  return e;
}

}  // namespace

cudaError_t launch_distill_short(const Ctx& c, const DistillArgs& a, int dtype, bool loss, bool grad) {
  return dtype == DH_BF16 ? run_short<__nv_bfloat16>(c, a, loss, grad) : run_short<float>(c, a, loss, grad);
}
bool distill_short_always(int N, int n_seg, bool step) { return n_seg <= DS_SEG_FEW && (step || N <= 512); }
bool distill_short(const DistillArgs& a, int num_sms, bool step) {
  if (distill_short_always(a.N, a.n_seg, step)) return true;
  return step ? a.n_seg <= DS_MAX_SEG && a.N >= num_sms : a.n_seg <= DS_SEG_FEW && a.N <= 8 * num_sms;
}
cudaError_t launch_distill_gather(const Ctx& c, const DistillArgs& a, int dtype) {
  return dtype == DH_BF16 ? run_gather<__nv_bfloat16>(c, a) : run_gather<float>(c, a);
}
cudaError_t launch_distill_dense(const Ctx& c, const DistillArgs& a, int dtype) {
  return dtype == DH_BF16 ? run_dense<__nv_bfloat16>(c, a) : run_dense<float>(c, a);
}
cudaError_t launch_distill_finish(const Ctx& c, const DistillArgs& a, int dtype, bool loss, bool grad) {
  return dtype == DH_BF16 ? run_finish<__nv_bfloat16>(c, a, loss, grad) : run_finish<float>(c, a, loss, grad);
}
cudaError_t launch_distill_grad(const Ctx& c, const DistillArgs& a, int dtype) {
  return dtype == DH_BF16 ? run_grad<__nv_bfloat16>(c, a) : run_grad<float>(c, a);
}

}  // namespace dh
