// Internal declarations of the operators between a row of logits and the head's next hidden rows
// (sample.cu, embed.cu, norm.cu; entry points in api_layers.cu).
//
// Programmatic dependent launch: a call's first kernel waits for the grid before it ahead of any access to
// memory, and the kernels inside a call let the next one of the call start early.  A call's last kernel lets
// nothing start before it has ended: the rescoring kernels load their hidden rows before their own wait, and
// those may be the rows that an embedding or a norm has just written.
#pragma once

#include "dh_internal.cuh"

namespace dh {

// Sampling (sample.cu).  Per-row settings, or one value for all rows where the pointer is null.
struct SampleArgs {
  const void* logits;  // [N] rows of `vocab`, stride ld elements
  long long ld;
  const float* u;  // [N]
  const float *temperature, *top_p, *min_p;
  const int32_t* top_k;
  float temperature0, top_p0, min_p0;
  int top_k0;
  int N, vocab;
  int32_t* token;
  float* prob;  // or null
  void* ws;
};
size_t sample_workspace(int N, int vocab, int dtype);
cudaError_t launch_sample(const Ctx& c, const SampleArgs& a, int dtype);

// Embedding (embed.cu).
struct EmbedArgs {
  const void* src;  // forward: the table; backward: the rows' gradients
  long long src_ld;
  void* dst;  // forward: the rows; backward: the table's gradient
  long long dst_ld;
  const int32_t* tokens;
  int N, vocab, d;
  float scale;
  bool accumulate;
  char* ws;
};
size_t embed_backward_workspace(int N, int vocab, int d, int dtype);
cudaError_t launch_embed(const Ctx& c, const EmbedArgs& a, int dtype);
cudaError_t launch_embed_backward(const Ctx& c, const EmbedArgs& a, int dtype);

// Layer norm (norm.cu).  Null: no weight, no bias, output not wanted.
struct NormArgs {
  const void* x;
  long long ld;
  const void *weight, *bias;
  float eps;
  void* y;  // forward: the normed rows; backward: the gradient of x
  long long y_ld;
  float2* stats_out;
  const float2* stats;
  const void* grad;
  long long grad_ld;
  void *grad_weight, *grad_bias;
  int N, d;
  int part_ld;  // columns of a block's sums in ws
  float* ws;
};
size_t norm_backward_workspace(int N, int d, int dtype);
cudaError_t launch_norm(const Ctx& c, const NormArgs& a, int dtype, int param_dtype);
cudaError_t launch_norm_backward(const Ctx& c, const NormArgs& a, int dtype, int param_dtype);

// Launches with programmatic stream serialization: the kernel may start while the grid before it ends, and
// waits for it by griddepcontrol.wait.  In clusters of `ranks` blocks (1: none).
template <class... P, class... A>
cudaError_t launch_clusters(const Ctx& c, const char* name, void (*kernel)(P...), unsigned ranks, dim3 grid, dim3 block,
                            size_t smem, A... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ranks;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cfg.attrs = at;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  prof_before(name, c.stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  prof_after(c.stream);
  return e;
}
template <class... P, class... A>
cudaError_t launch_pdl(const Ctx& c, const char* name, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                       A... args) {
  return launch_clusters(c, name, kernel, 1, grid, block, smem, args...);
}

// ------------------------------------------------------------------ thread-block clusters

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// The word at `p` of this block's shared memory, in block `rank` of the cluster.
__device__ __forceinline__ uint32_t ld_cluster(const uint32_t* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_cluster(const uint4* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(r)
               : "memory");
  return v;
}

// ------------------------------------------------------------------ rows of hidden states

// Which columns of a row a thread holds: NV vectors of PER16 of them.  A warp's columns are contiguous, so that a
// thread's vectors lie at constant distances.  VEC, for rows of whole vectors that start on 16 bytes: a vector is
// adjacent columns, in one access, and a warp's vectors v stand together.  Otherwise a thread has every 32nd column
// of its warp's, so that neighbouring threads access neighbouring elements whatever the row's alignment.  Columns
// past the row's end read as 0 and are not written.
template <typename T, bool VEC, int NV = 1>
struct Cols {
  static constexpr int PER = Elem<T>::PER16;
  static constexpr int WARP = 32 * NV * PER;  // columns of a warp
  __device__ __forceinline__ static int col(int thread, int v, int e) {
    return (thread >> 5) * WARP + (VEC ? (v * 32 + (thread & 31)) * PER + e : (v * PER + e) * 32 + (thread & 31));
  }
  __device__ __forceinline__ static uint4 load(const T* row, int thread, int v, int d) {
    if constexpr (VEC) {
      const int id = col(thread, v, 0);
      return id < d ? *reinterpret_cast<const uint4*>(row + id) : make_uint4(0u, 0u, 0u, 0u);
    } else {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const int id = col(thread, v, e);
        if (id < d) {
          if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(row[id]);
          else w[e / 2] |= (uint32_t)__bfloat16_as_ushort(row[id]) << (16 * (e & 1));
        }
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ static void store(T* row, int thread, int v, int d, const uint4& u) {
    if constexpr (VEC) {
      const int id = col(thread, v, 0);
      if (id < d) *reinterpret_cast<uint4*>(row + id) = u;
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const int id = col(thread, v, e);
        if (id < d) {
          if constexpr (sizeof(T) == 4) row[id] = __uint_as_float(w[e]);
          else row[id] = __ushort_as_bfloat16((unsigned short)(w[e / 2] >> (16 * (e & 1))));
        }
      }
    }
  }
};

// Whether rows of d elements at p, `ld` elements apart, are whole vectors that start on 16 bytes.
inline bool whole_vectors(const void* p, long long ld, long long rows, int d, int elem) {
  return d * (long long)elem % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 &&
         (rows <= 1 || ld * elem % 16 == 0);
}

// PER16 fp32 values, each rounded once to T.
template <typename T>
__device__ __forceinline__ uint4 round_vec(const float* z) {
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

}  // namespace dh
