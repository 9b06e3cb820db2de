// Distillation from a teacher's top logits: the loss of a student's rows of logits and its gradient
// (definitions at dh_distill_topk in dh.h).
//
// With p = softmax(y / T) over the teacher's entries and q = softmax(z / T) over the vocabulary,
//   loss = T^2 sum_k p_k (log p_k - log q[id_k]),   dz[v] = g T (q[v] - sum of the p_k with id_k = v).
// Only the normaliser of q needs the whole row; the entries are a sparse correction of the dense
// term g T q.  So the loss reads the row once (row_stats.cu) and finishes with K gathered logits,
// and the gradient reads it once and writes it once: both are bound by HBM.
//
// k_distill_loss: one block per row; the segments' pairs -> (max, sum), the teacher's softmax, the
//   loss.
// k_distill_grad: `splits` blocks per row, each streaming its part of the row.  The logits of the
//   part's entries are read before the dense pass writes anything (the gradient may overwrite the
//   logits); after the pass the same block writes the entries' values, one writer per id: the first
//   entry of an id adds up the others' p in order, so repeated ids repeat bit for bit.
#include "rows.cuh"

namespace dh {
namespace {

constexpr int DL_THREADS = 128;
constexpr int DG_THREADS = 256;
constexpr int DG_UNROLL = 4;

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

// T^2 sum_k p_k (log p_k - log q_k) of one row, by the whole block (every thread gets it).
template <typename T, int NT>
__device__ __forceinline__ float row_loss(const T* row, const float* __restrict__ y, int nk, const Teacher& t,
                                          const int32_t* s_id, const float* s_p, float m, float sum, float temperature,
                                          float inv_t, float* red) {
  const float log_sum = logf(sum);
  float part = 0.f;
  for (int k = threadIdx.x; k < nk; k += NT) {
    const float p = s_p[k];
    if (s_id[k] < 0 || p == 0.f) continue;  // 0 log 0 = 0
    const float z = Elem<T>::to_f(row[s_id[k]]);
    const float log_q = m == -INFINITY ? -INFINITY : (z - m) * inv_t - log_sum;
    part += p * (((__ldg(y + k) - t.top) * inv_t - t.log_total) - log_q);
  }
  return temperature * temperature * block_sum<NT>(part, red);
}

template <typename T>
__global__ void __launch_bounds__(DL_THREADS) k_distill_loss(DistillArgs a) {
  __shared__ int32_t s_id[DH_MAX_K];
  __shared__ float s_p[DH_MAX_K];
  __shared__ float red[DL_THREADS / 32];
  __shared__ float s_m, s_s;
  const int row = blockIdx.x;
  const int32_t* idx = a.idx + (size_t)row * a.K;
  const float* y = a.teacher + (size_t)row * a.K;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int nk = a.n_valid ? min(max(__ldg(a.n_valid + row), 0), a.K) : a.K;
  if (threadIdx.x < 32) {
    float m;
    Sum2 s;
    row_combine(a.seg + (size_t)row * a.n_seg, a.n_seg, a.inv_t, &m, &s);
    if (threadIdx.x == 0) {
      s_m = m;
      s_s = s.hi + s.lo;
      if (a.stats_out) a.stats_out[row] = make_float2(m, s_s);
    }
  }
  const Teacher t = teacher_row<DL_THREADS>(idx, y, nk, a.vocab, a.inv_t, s_id, s_p, red);
  __syncthreads();
  float loss = 0.f;
  if (t.any)
    loss = row_loss<T, DL_THREADS>(static_cast<const T*>(a.logits) + (size_t)row * a.ld, y, nk, t, s_id, s_p, s_m, s_s,
                                   a.temperature, a.inv_t, red);
  if (threadIdx.x == 0) a.loss_out[row] = loss;
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

// a 2^((z - m) c) for the elements of a vector, rounded once to the logits' type.
template <typename T>
__device__ __forceinline__ uint4 grad_vec(const uint4& u, float m, float c, float a) {
  constexpr int PER = Elem<T>::PER16;
  float z[PER];
  Elem<T>::unpack(u, z);
#pragma unroll
  for (int e = 0; e < PER; ++e) z[e] = a * row_ex2((z[e] - m) * c);
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (sizeof(T) == 4) {
      w[q] = __float_as_uint(z[q]);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(z[2 * q], z[2 * q + 1]);
      w[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  const float aq = t.log_total != t.log_total ? t.log_total : (nothing ? 0.f : g / sum), mm = nothing ? 0.f : m;
  const T* zv = z + pre;
  const bool same = ((reinterpret_cast<uintptr_t>(zv)) & 15u) == 0;
  auto scalar = [&](int i) { out[i] = Elem<T>::from_f(aq * row_ex2((Elem<T>::to_f(z[i]) - mm) * a.c)); };
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
      if (jj < vhi) st16(out + pre + (long long)jj * PER, grad_vec<T>(u[q], mm, a.c, aq));
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
    if (first) out[id] = Elem<T>::from_f(aq * row_ex2((s_z[k] - mm) * a.c) - g * p);
  }
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
cudaError_t run_loss(const Ctx& c, const DistillArgs& a) {
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = pdl_config(c, (unsigned)a.N, DL_THREADS, &at);
  prof_before("distill_loss", c.stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_distill_loss<T>, a);
  prof_after(c.stream);
  return e;
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

}  // namespace

cudaError_t launch_distill_loss(const Ctx& c, const DistillArgs& a, int dtype) {
  return dtype == DH_BF16 ? run_loss<__nv_bfloat16>(c, a) : run_loss<float>(c, a);
}
cudaError_t launch_distill_grad(const Ctx& c, const DistillArgs& a, int dtype) {
  return dtype == DH_BF16 ? run_grad<__nv_bfloat16>(c, a) : run_grad<float>(c, a);
}

}  // namespace dh
