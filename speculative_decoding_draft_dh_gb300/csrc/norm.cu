// Layer norm over the last dimension, and its gradients (definitions at dh_layer_norm and
// dh_layer_norm_backward in dh.h).
//
// The bound is HBM: a row is read once, held in registers, and written once.  A row belongs to a warp (up to 128
// vectors of 16 bytes) or to a block; the groups walk over the rows and load their next row before they reduce
// the present one.
// Forward: the mean first, then the sums of x - mean and of its square, so that the variance loses nothing to a
// mean far from 0 (the two-pass form with the correction of Chan, Golub and LeVeque).
// Backward: with xhat = (x - mean) rstd and h = g w,
//   dx = rstd (h - mean(h) - xhat mean(h xhat)),   dw = sum_n g xhat,   db = sum_n g.
// A thread keeps its columns over all rows that its group walks, so dw and db are summed in its registers;
// blocks leave their sums in the workspace and a second kernel adds them in order.
// Rows of more than NM_HELD columns are read again for each step instead, by k_norm_wide and
// k_norm_backward_wide, and k_norm_columns sums their dw and db.
#include "layers.cuh"

namespace dh {
namespace {

constexpr int NM_HELD = 8192;  // columns of a row that registers hold

// N parameters of type P at the columns of Cols<T, VEC>'s vector v (0 past the end).
template <typename P, int N>
struct Params {
  uint4 raw[N * sizeof(P) / 16];
  __device__ __forceinline__ void unpack(float* z) const {
    constexpr int PER = Elem<P>::PER16;
#pragma unroll
    for (int q = 0; q < N / PER; ++q) Elem<P>::unpack(raw[q], z + q * PER);
  }
};
template <typename T, typename P, bool VEC>
__device__ __forceinline__ void load_params(Params<P, Elem<T>::PER16>& u, const P* p, int thread, int width, int v,
                                            int d) {
  constexpr int N = Elem<T>::PER16, PER = Elem<P>::PER16;
  if constexpr (VEC) {
    const int id = Cols<T, VEC>::col(thread, width, v, 0);
#pragma unroll
    for (int q = 0; q < N / PER; ++q)
      u.raw[q] = id < d ? __ldg(reinterpret_cast<const uint4*>(p + id) + q) : make_uint4(0u, 0u, 0u, 0u);
  } else {
    float z[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int id = Cols<T, VEC>::col(thread, width, v, e);
      z[e] = id < d ? Elem<P>::to_f(p[id]) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < N / PER; ++q) u.raw[q] = round_vec<P>(z + q * PER);  // exact: they are P values
  }
}

// Sums of a and b over the row's group, a warp or the block; every thread gets them.  `turn` alternates, so that
// one barrier per call is enough.
template <bool WARP>
__device__ __forceinline__ float2 group_sum(float a, float b, float2 (*sh)[32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  if (WARP) return make_float2(a, b);
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

constexpr int NF_WARPS = 4;  // rows of a block where a row belongs to a warp

template <typename T, typename P, int NV, bool WARP, bool VEC>
__global__ void __launch_bounds__(WARP ? 32 * NF_WARPS : 1024) k_norm(NormArgs a) {
  using C = Cols<T, VEC>;
  constexpr int PER = C::PER;
  __shared__ float2 sh[2][32];
  const int me = WARP ? (threadIdx.x & 31) : threadIdx.x, width = WARP ? 32 : blockDim.x;
  const long long groups = WARP ? (long long)gridDim.x * NF_WARPS : gridDim.x;
  long long n = WARP ? (long long)blockIdx.x * NF_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  const float inv_d = 1.f / (float)a.d;
  int turn = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n >= a.N) return;  // a whole group
  uint4 u[NV], next[NV];
  Params<P, PER> w[NV], b[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) u[v] = C::load(x + n * a.ld, me, width, v, a.d);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (a.weight) load_params<T, P, VEC>(w[v], static_cast<const P*>(a.weight), me, width, v, a.d);
    if (a.bias) load_params<T, P, VEC>(b[v], static_cast<const P*>(a.bias), me, width, v, a.d);
  }
  for (; n < a.N; n += groups) {
    if (n + groups < a.N) {
#pragma unroll
      for (int v = 0; v < NV; ++v) next[v] = C::load(x + (n + groups) * a.ld, me, width, v, a.d);
    }
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float z[PER];
      Elem<T>::unpack(u[v], z);
#pragma unroll
      for (int e = 0; e < PER; ++e) s += z[e];
    }
    const float mean0 = group_sum<WARP>(s, 0.f, sh, turn).x * inv_d;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float z[PER];
      Elem<T>::unpack(u[v], z);
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const float t = C::col(me, width, v, e) < a.d ? z[e] - mean0 : 0.f;
        s1 += t;
        s2 = fmaf(t, t, s2);
      }
    }
    const Moments q = moments(mean0, group_sum<WARP>(s1, s2, sh, turn), inv_d, a.eps);
    if (a.stats_out && me == 0) a.stats_out[n] = make_float2(q.mean0 + q.delta, q.rstd);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float z[PER], wv[PER], bv[PER];
      Elem<T>::unpack(u[v], z);
      if (a.weight) w[v].unpack(wv);
      if (a.bias) b[v].unpack(bv);
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        z[e] = ((z[e] - q.mean0) - q.delta) * q.rstd;
        if (a.weight) z[e] = a.bias ? fmaf(z[e], wv[e], bv[e]) : z[e] * wv[e];
        else if (a.bias) z[e] += bv[e];
      }
      C::store(y + n * a.y_ld, me, width, v, a.d, round_vec<T>(z));
      u[v] = next[v];
    }
  }
}

constexpr int NB_WARPS = 8;  // backward: rows of a block where a row belongs to a warp
constexpr int NB_THREADS = 512;

template <typename T, typename P, int NV, bool WARP, bool VEC>
__global__ void __launch_bounds__(WARP ? 32 * NB_WARPS : NB_THREADS) k_norm_backward(NormArgs a, bool sums) {
  using C = Cols<T, VEC>;
  constexpr int PER = C::PER;
  __shared__ float2 sh[2][32];
  __shared__ float s_sum[WARP ? 2 * 32 * NV * PER : 1];
  const int me = WARP ? (threadIdx.x & 31) : threadIdx.x, width = WARP ? 32 : blockDim.x;
  const long long groups = WARP ? (long long)gridDim.x * NB_WARPS : gridDim.x;
  const T* x = static_cast<const T*>(a.x);
  const T* g = static_cast<const T*>(a.grad);
  T* dx = static_cast<T*>(a.y);
  const float inv_d = 1.f / (float)a.d;
  int turn = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (sums) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel follows
  long long n = WARP ? (long long)blockIdx.x * NB_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  uint4 u[NV], h[NV], un[NV], hn[NV];
  Params<P, PER> w[NV];
  float dw[NV][PER], db[NV][PER];
  float2 st = make_float2(0.f, 0.f), stn = st;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int e = 0; e < PER; ++e) dw[v][e] = db[v][e] = 0.f;
    if (n < a.N) {
      u[v] = C::load(x + n * a.ld, me, width, v, a.d);
      h[v] = C::load(g + n * a.grad_ld, me, width, v, a.d);
    }
    if (a.weight) load_params<T, P, VEC>(w[v], static_cast<const P*>(a.weight), me, width, v, a.d);
  }
  if (n < a.N) st = __ldg(a.stats + n);
  for (; n < a.N; n += groups) {
    const long long m = n + groups;
    if (m < a.N) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        un[v] = C::load(x + m * a.ld, me, width, v, a.d);
        hn[v] = C::load(g + m * a.grad_ld, me, width, v, a.d);
      }
      stn = __ldg(a.stats + m);
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float z[PER], q[PER], wv[PER];
      Elem<T>::unpack(u[v], z);
      Elem<T>::unpack(h[v], q);
      if (a.weight) w[v].unpack(wv);
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        // past the row's end g is 0, and so is what it is multiplied with (the row's statistics may be NaN)
        const float hat = C::col(me, width, v, e) < a.d ? (z[e] - st.x) * st.y : 0.f;
        dw[v][e] = fmaf(q[e], hat, dw[v][e]);
        db[v][e] += q[e];
        const float t = a.weight ? q[e] * wv[e] : q[e];
        s1 += t;
        s2 = fmaf(t, hat, s2);
      }
    }
    if (dx) {
      const float2 c = group_sum<WARP>(s1, s2, sh, turn);
      const float c1 = c.x * inv_d, c2 = c.y * inv_d;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float z[PER], q[PER], wv[PER];
        Elem<T>::unpack(u[v], z);
        Elem<T>::unpack(h[v], q);
        if (a.weight) w[v].unpack(wv);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const float hat = (z[e] - st.x) * st.y;
          const float t = a.weight ? q[e] * wv[e] : q[e];
          z[e] = st.y * fmaf(-hat, c2, t - c1);
        }
        C::store(dx + n * a.y_ld, me, width, v, a.d, round_vec<T>(z));
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      u[v] = un[v];
      h[v] = hn[v];
    }
    st = stn;
  }
  if (!sums) return;
  float* part = a.ws + (long long)blockIdx.x * 2 * a.d;
  if (WARP) {
    // the warps add theirs one after another
    for (int r = 0; r < NB_WARPS; ++r) {
      if ((int)(threadIdx.x >> 5) == r) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            float* q = s_sum + ((v * PER + e) * 32 + me) * 2;
            q[0] = (r ? q[0] : 0.f) + dw[v][e];
            q[1] = (r ? q[1] : 0.f) + db[v][e];
          }
      }
      __syncthreads();
    }
    if (threadIdx.x >= 32) return;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int id = C::col(me, width, v, e);
      const float* q = s_sum + ((v * PER + e) * 32 + me) * 2;
      if (id < a.d) {
        part[id] = WARP ? q[0] : dw[v][e];
        part[a.d + id] = WARP ? q[1] : db[v][e];
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
    const float mean0 = group_sum<false>(s, 0.f, sh, turn).x * inv_d;
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < a.d; i += NW_THREADS) {
      const float t = Elem<T>::to_f(x[i]) - mean0;
      s1 += t;
      s2 = fmaf(t, t, s2);
    }
    const Moments q = moments(mean0, group_sum<false>(s1, s2, sh, turn), inv_d, a.eps);
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
__global__ void __launch_bounds__(NW_THREADS) k_norm_backward_wide(NormArgs a, bool sums) {
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
    const float2 c = group_sum<false>(s1, s2, sh, turn);
    const float c1 = c.x * inv_d, c2 = c.y * inv_d;
    for (int i = threadIdx.x; i < a.d; i += NW_THREADS) {
      const float t = terms(i, &hat);
      dx[i] = Elem<T>::from_f(st.y * fmaf(-hat, c2, t - c1));
    }
  }
}

// dw and db of a tile of columns over a share of the rows.
constexpr int NC_THREADS = 256;
template <typename T>
__global__ void __launch_bounds__(NC_THREADS) k_norm_columns(NormArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel follows
  const int col = blockIdx.x * NC_THREADS + threadIdx.x;
  if (col >= a.d) return;
  const T* x = static_cast<const T*>(a.x) + col;
  const T* g = static_cast<const T*>(a.grad) + col;
  float dw = 0.f, db = 0.f;
  for (long long n = blockIdx.y; n < a.N; n += gridDim.y) {
    const float2 st = __ldg(a.stats + n);
    const float q = Elem<T>::to_f(g[n * a.grad_ld]);
    dw = fmaf(q, (Elem<T>::to_f(x[n * a.ld]) - st.x) * st.y, dw);
    db += q;
  }
  float* part = a.ws + (long long)blockIdx.y * 2 * a.d;
  part[col] = dw;
  part[a.d + col] = db;
}

// The blocks' sums, added in a fixed order and rounded once.
constexpr int NJ_COLS = 32, NJ_ROWS = 16;
template <typename P>
__global__ void __launch_bounds__(NJ_COLS * NJ_ROWS) k_norm_join(NormArgs a, int parts) {
  __shared__ float sh[NJ_ROWS][NJ_COLS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int col = blockIdx.x * NJ_COLS + (threadIdx.x & 31), row = threadIdx.x >> 5;
  P* out = static_cast<P*>(blockIdx.y ? a.grad_bias : a.grad_weight);
  if (!out) return;
  float s = 0.f;
  if (col < a.d)
    for (int i = row; i < parts; i += NJ_ROWS) s += a.ws[((long long)i * 2 + blockIdx.y) * a.d + col];
  sh[row][threadIdx.x & 31] = s;
  __syncthreads();
  if (row == 0 && col < a.d) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < NJ_ROWS; ++r) t += sh[r][threadIdx.x];
    out[col] = Elem<P>::from_f(t);
  }
}

constexpr int NM_PARTS = 512;  // blocks that leave sums, at most

int round32(int x) { return (x + 31) / 32 * 32; }
unsigned least(long long a, long long b) { return (unsigned)(a < b ? a : b); }

template <typename T, typename P, bool VEC>
cudaError_t run_norm(const Ctx& c, const NormArgs& a) {
  constexpr int PER = Elem<T>::PER16;
  const int nvec = (a.d + PER - 1) / PER;
  auto go = [&](auto* kernel, unsigned grid, unsigned threads) {
    return launch_pdl(c, "norm", kernel, dim3(grid), dim3(threads), 0, a);
  };
  const unsigned by_warp = least(((long long)a.N + NF_WARPS - 1) / NF_WARPS, 12LL * c.num_sms);
  if (nvec <= 32) return go(k_norm<T, P, 1, true, VEC>, by_warp, 32 * NF_WARPS);
  if (nvec <= 128) return go(k_norm<T, P, 4, true, VEC>, by_warp, 32 * NF_WARPS);
  const int nv = nvec <= 640 ? 1 : 2, threads = round32((nvec + nv - 1) / nv);
  const unsigned by_block = least(a.N, (long long)c.num_sms * (2048 / threads > 8 ? 8 : 2048 / threads));
  return nv == 1 ? go(k_norm<T, P, 1, false, VEC>, by_block, (unsigned)threads)
                 : go(k_norm<T, P, 2, false, VEC>, by_block, (unsigned)threads);
}

template <typename T, typename P, bool VEC>
cudaError_t run_norm_backward(const Ctx& c, const NormArgs& a, bool sums, int* parts) {
  constexpr int PER = Elem<T>::PER16;
  const int nvec = (a.d + PER - 1) / PER;
  auto go = [&](auto* kernel, unsigned grid, unsigned threads) {
    *parts = (int)grid;
    return launch_pdl(c, "norm_backward", kernel, dim3(grid), dim3(threads), 0, a, sums);
  };
  const unsigned by_warp = least(((long long)a.N + NB_WARPS - 1) / NB_WARPS, least(NM_PARTS, 3LL * c.num_sms));
  if (nvec <= 32) return go(k_norm_backward<T, P, 1, true, VEC>, by_warp, 32 * NB_WARPS);
  const int nv = nvec <= NB_THREADS ? 1 : nvec <= 2 * NB_THREADS ? 2 : 4, threads = round32((nvec + nv - 1) / nv);
  const unsigned by_block = least(a.N, least(NM_PARTS, (long long)c.num_sms * (1024 / threads > 8 ? 8 : 1024 / threads)));
  if (nv == 1) return go(k_norm_backward<T, P, 1, false, VEC>, by_block, (unsigned)threads);
  if (nv == 2) return go(k_norm_backward<T, P, 2, false, VEC>, by_block, (unsigned)threads);
  if constexpr (sizeof(T) == 4) return go(k_norm_backward<T, P, 4, false, VEC>, by_block, (unsigned)threads);
  return cudaErrorInvalidValue;  // not reached: 8192 bf16 columns are 1024 vectors
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
cudaError_t pick_backward(const Ctx& c, const NormArgs& a) {
  const bool sums = a.grad_weight || a.grad_bias;
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (a.N == 0) {
    // sums of no rows: the joining kernel writes zeros
  } else if (a.d <= NM_HELD) {
    const bool vec = params16(a.weight, nullptr) && whole_vectors(a.x, a.ld, a.N, a.d, sizeof(T)) &&
                     whole_vectors(a.grad, a.grad_ld, a.N, a.d, sizeof(T)) &&
                     (!a.y || whole_vectors(a.y, a.y_ld, a.N, a.d, sizeof(T)));
    e = vec ? run_norm_backward<T, P, true>(c, a, sums, &parts) : run_norm_backward<T, P, false>(c, a, sums, &parts);
  } else {
    // the columns' sums first: the gradient may overwrite the rows
    if (sums) {
      const int tiles = (a.d + NC_THREADS - 1) / NC_THREADS, shares = 8 * c.num_sms / tiles;
      parts = (int)least(a.N, least(NM_PARTS, shares < 1 ? 1 : shares));
      e = launch_pdl(c, "norm_columns", k_norm_columns<T>, dim3((unsigned)tiles, (unsigned)parts), dim3(NC_THREADS), 0,
                     a);
    }
    if (e == cudaSuccess && a.y)
      e = launch_pdl(c, "norm_backward", k_norm_backward_wide<T, P>, dim3(least(a.N, 2LL * c.num_sms)),
                     dim3(NW_THREADS), 0, a, sums);
  }
  if (e != cudaSuccess || !sums) return e;
  return launch_pdl(c, "norm_join", k_norm_join<P>, dim3((unsigned)((a.d + NJ_COLS - 1) / NJ_COLS), 2u),
                    dim3(NJ_COLS * NJ_ROWS), 0, a, parts);
}

}  // namespace

size_t norm_backward_workspace(int N, int d, int) {
  return WS_HEADER + align_up((size_t)(N < NM_PARTS ? N : NM_PARTS) * 2 * d * sizeof(float), 256);
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
