// Embedding lookup with scaling, and the table's gradient by sorted tokens (definitions at dh_embed and
// dh_embed_backward in dh.h).
//
// Lookup: out[n] = scale table[token[n]].  Nothing but the copy's traffic: a thread moves VECS vectors of 16
// bytes, all loads issued before the first store.  32768 rows of 5120 bf16 in 76 us: 455 MB at 6.0 TB/s.
//
// Gradient: grad[v] = scale sum over the n with token[n] = v, in fp32.  The positions are first sorted by
// (token, n), so that a row's terms stand together and are added in one fixed order, without atomics on
// values:
//   k_token_sort   a stable radix sort of the N (token, n) pairs by one cluster, in a single launch; also marks
//                  the tokens that occur in a bitmap
//   k_embed_grad   blocks over chunks of the sorted pairs, each for a tile of columns: a run of one token that
//                  lies within its chunk is summed and written; of a run that leaves its chunk, the part is
//                  written to the workspace.  More blocks write the zeros of the rows that do not occur.
//   k_embed_join   adds the parts of the runs that span chunks, in order.
// The split by chunks of pairs, not by rows, keeps the work even however often one token comes.  The bound is HBM,
// most of it the zeros of the rows that do not occur: 32768 tokens of 5120 bf16 into 151936 rows, 1.9 GB, in 287 us
// (6.5 TB/s), of which the sort takes 20.  Of fewer tokens the sort is the larger part: 20011 of 1001 fp32 into 4096
// rows 41 us, sort 16.
#include <type_traits>

#include "layers.cuh"
#include "rows.cuh"

namespace dh {
namespace {

constexpr int EM_THREADS = 256;
// 4 for long calls: 32768 rows of 5120 bf16 75 us, 79 with 2, 78 with 8.  1 where those are fewer than EM_FEW blocks per
// SM: 8 rows 1.2 us, 1.8 with 4; 1000 rows 3.1 and 3.4; 2000 rows 6.2 and 5.4.
constexpr int EM_VECS = 4, EM_FEW = 8;

// Pieces of a row that is written: its 16-byte words in memory, of which the first and the last may hold elements of
// its neighbours, so that what is written is whole words whatever the row's alignment.  Piece g starts at column
// g PER - lead, lead being the elements between the row's start and the word's.  (32768 rows of 5119 bf16: 122 us, and
// 345 element by element; the gradient's sums go by elements, since pieces that hang on each token's row took 76 us
// where elements take 41, 20011 fp32 rows of 1001.)
template <typename T>
__device__ __forceinline__ int lead(const T* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}
inline int pieces(int d, int per) { return (d + per - 1) / per + 1; }
// Columns [col, col + PER) of a row of any alignment, 0 outside [0, d).
template <typename T>
__device__ __forceinline__ uint4 load_piece(const T* row, int col, int d) {
  constexpr int PER = Elem<T>::PER16;
  if (col >= 0 && col + PER <= d) return ld16_any(row + col);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (col < d && col + PER > 0) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      if (col + e >= 0 && col + e < d) {
        const uint32_t b = elem_bits(row[col + e]);
        if (sizeof(T) == 4) w[e] = b;
        else w[e / 2] |= b << (16 * (e & 1));
      }
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void store_piece(T* row, int col, int d, const uint4& u) {
  constexpr int PER = Elem<T>::PER16;
  if (col >= 0 && col + PER <= d) {
    *reinterpret_cast<uint4*>(row + col) = u;
  } else if (col < d && col + PER > 0) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      if (col + e < 0 || col + e >= d) continue;
      if constexpr (sizeof(T) == 4) row[col + e] = __uint_as_float(w[e]);
      else row[col + e] = __ushort_as_bfloat16((unsigned short)(w[e / 2] >> (16 * (e & 1))));
    }
  }
}

// A unit is 16 bytes of a row, with all rows starting on 16 bytes (VEC), else a piece; `units` of them make a row.
template <typename T, bool VEC, int VECS>
__global__ void __launch_bounds__(EM_THREADS) k_embed(EmbedArgs a, unsigned units) {
  constexpr int PER = Elem<T>::PER16;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const T* table = static_cast<const T*>(a.src);
  T* out = static_cast<T*>(a.dst);
  const unsigned long long items = (unsigned long long)a.N * units;
  const unsigned long long i0 = (unsigned long long)blockIdx.x * (EM_THREADS * VECS) + threadIdx.x;
  uint4 x[VECS];
  int row[VECS], at[VECS];
  float by[VECS];  // the scale; 1 where padding is: its zeros stay zeros whatever the scale
#pragma unroll
  for (int q = 0; q < VECS; ++q) {
    const unsigned long long i = i0 + q * EM_THREADS;
    row[q] = -1;
    by[q] = 1.f;
    if (i < items) {
      const unsigned long long r = i / units;
      row[q] = (int)r;
      at[q] = (int)(i - r * units) * PER;
      if (!VEC) at[q] -= lead(out + r * a.dst_ld);
      const int t = __ldg(a.tokens + r);
      x[q] = make_uint4(0u, 0u, 0u, 0u);
      if (t >= 0 && t < a.vocab) {
        by[q] = a.scale;
        const T* from = table + (long long)t * a.src_ld;
        x[q] = VEC ? *reinterpret_cast<const uint4*>(from + at[q]) : load_piece(from, at[q], a.d);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < VECS; ++q) {
    if (row[q] < 0) continue;
    if (a.scale != 1.f) {
      float z[PER];
      Elem<T>::unpack(x[q], z);
#pragma unroll
      for (int e = 0; e < PER; ++e) z[e] *= by[q];
      x[q] = round_vec<T>(z);
    }
    T* to = out + row[q] * a.dst_ld;
    if (VEC) *reinterpret_cast<uint4*>(to + at[q]) = x[q];
    else store_piece(to, at[q], a.d, x[q]);
  }
}

// ------------------------------------------------------------------ sorting the tokens

constexpr int TS_THREADS = 1024;
constexpr int TS_WARPS = TS_THREADS / 32;
constexpr int TS_BITS = 9;   // at most, per pass
constexpr int TS_ITEMS = 8;  // rows of 32 pairs of a warp at a time
constexpr int TS_RANKS = 8;  // blocks of the cluster, at most
constexpr int TS_FEW = 2048;  // tokens that one block sorts, at most

// The lanes whose digit is this lane's, among those that have one.  By a ballot per bit: a match instruction takes
// an SM many times as long (a sort of 32768 tokens 27 us with it).
template <int BITS>
__device__ __forceinline__ uint32_t same_digit(uint32_t dg, bool on) {
  uint32_t same = __ballot_sync(0xFFFFFFFFu, on);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const bool bit = (dg >> b) & 1u;
    const uint32_t ones = __ballot_sync(0xFFFFFFFFu, bit);
    same &= bit ? ones : ~ones;
  }
  return same;
}

// Sorts (token, n) by token, stable in n, into buf0 after an odd number of passes, else buf1; tokens outside
// [0, vocab) get the key vocab and so come last.  A least-significant-digit radix sort: each warp owns a contiguous
// run of pairs, counts its digits, and after an exclusive scan over (digit, block, warp) places its pairs in order.
// What bounds it are latencies: of the passes, as few as digits of 9 bits allow (the counts of 32 warps fit shared
// memory), and of memory, so that a warp's loads are issued TS_ITEMS at a time, and up to that many pairs per lane
// stay in registers between counting and placing.  One cluster, since a pass then costs two cluster barriers and no
// launch: 32768 tokens of 18 bits in 22 us by 8 blocks, in 107 by one; 300 tokens 1.5 us less by one block.
template <int BITS>
__global__ void __launch_bounds__(TS_THREADS) k_token_sort(const int32_t* __restrict__ tokens, int N, int vocab,
                                                           int passes, uint2* __restrict__ buf0,
                                                           uint2* __restrict__ buf1, uint32_t* __restrict__ present) {
  constexpr int NB = 1 << BITS;
  extern __shared__ uint32_t cnt[];  // [warp][digit]
  __shared__ uint32_t s_total[NB], s_base[NB], s_scan[TS_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), ranks = cluster_size(), under = (1u << lane) - 1u;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int words = (vocab + 31) / 32;
  for (int i = rank * TS_THREADS + threadIdx.x; i < words; i += ranks * TS_THREADS) present[i] = 0u;
  // pairs of a warp: a multiple of 32, contiguous
  const unsigned warps = ranks * TS_WARPS;
  const long long per_warp = ((long long)N + 32LL * warps - 1) / (32LL * warps) * 32;
  const long long w0 = per_warp * (rank * TS_WARPS + warp);
  const int p0 = (int)(w0 < N ? w0 : N), p1 = (int)(w0 + per_warp < N ? w0 + per_warp : N);
  const bool once = per_warp <= 32 * TS_ITEMS;
  uint32_t* mine = cnt + warp * NB;
  uint2 x[TS_ITEMS];
  for (int pass = 0; pass < passes; ++pass) {
    const uint2* src = (pass & 1) ? buf0 : buf1;
    uint2* dst = (pass & 1) ? buf1 : buf0;
    const int sh = pass * BITS;
    // the pairs from i on, TS_ITEMS rows of 32; past the end the digit is none
    auto load = [&](int i) {
#pragma unroll
      for (int q = 0; q < TS_ITEMS; ++q) {
        const int at = i + q * 32 + lane;
        x[q] = make_uint2(0xFFFFFFFFu, 0u);
        if (at < p1) {
          if (pass == 0) {
            const int t = __ldg(tokens + at);
            x[q] = make_uint2((uint32_t)t < (uint32_t)vocab ? (uint32_t)t : (uint32_t)vocab, (uint32_t)at);
          } else {
            x[q] = __ldcg(src + at);
          }
        }
      }
    };
    for (int i = threadIdx.x; i < NB * TS_WARPS / 4; i += TS_THREADS)
      reinterpret_cast<uint4*>(cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p0 < p1) load(p0);
    __syncthreads();
    for (int i = p0; i < p1; i += 32 * TS_ITEMS) {
      if (i > p0) load(i);
#pragma unroll
      for (int q = 0; q < TS_ITEMS; ++q) {
        if (i + q * 32 >= p1) break;
        const bool on = x[q].x != 0xFFFFFFFFu;
        const uint32_t dg = (x[q].x >> sh) & (NB - 1u), same = same_digit<BITS>(dg, on);
        if (on && (same & under) == 0) mine[dg] += __popc(same);
        __syncwarp();
      }
    }
    __syncthreads();
    // per digit: the warps' counts to exclusive sums, and the block's total
    for (int b = threadIdx.x; b < NB; b += TS_THREADS) {
      uint32_t s = 0;
#pragma unroll
      for (int w0 = 0; w0 < TS_WARPS; w0 += 8) {
        uint32_t c[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) c[w] = cnt[(w0 + w) * NB + b];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          cnt[(w0 + w) * NB + b] = s;
          s += c[w];
        }
      }
      s_total[b] = s;
    }
    cluster_sync();
    // the digit's first place of this block: lower digits of all blocks, the same digit of lower blocks
    uint32_t all = 0, before = 0;
    if (threadIdx.x < NB) {
#pragma unroll
      for (uint32_t r = 0; r < TS_RANKS; ++r) {
        const uint32_t c = r < ranks ? ld_cluster(s_total + threadIdx.x, r) : 0u;
        all += c;
        if (r < rank) before += c;
      }
    }
    uint32_t inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    if (threadIdx.x < NB) {
      uint32_t base = inc - all + before;
      for (int w = 0; w < warp; ++w) base += s_scan[w];
      s_base[threadIdx.x] = base;
    }
    __syncthreads();
    for (int i = p0; i < p1; i += 32 * TS_ITEMS) {
      if (!once) load(i);
#pragma unroll
      for (int q = 0; q < TS_ITEMS; ++q) {
        if (i + q * 32 >= p1) break;
        const bool on = x[q].x != 0xFFFFFFFFu;
        const uint32_t dg = (x[q].x >> sh) & (NB - 1u), same = same_digit<BITS>(dg, on);
        const uint32_t below = same & under;
        if (on) dst[s_base[dg] + mine[dg] + __popc(below)] = x[q];
        __syncwarp();
        if (on && below == 0) mine[dg] += __popc(same);
        __syncwarp();
      }
    }
    // the pairs are in place for the whole cluster, and the totals have been read
    cluster_sync();
  }
  // the tokens that occur, each once: where a run starts
  const uint2* sorted = (passes & 1) ? buf0 : buf1;
  for (int i = rank * TS_THREADS + threadIdx.x; i < N; i += ranks * TS_THREADS) {
    const uint32_t t = __ldcg(sorted + i).x;
    if (t < (uint32_t)vocab && (i == 0 || __ldcg(sorted + i - 1).x != t)) atomicOr(present + (t >> 5), 1u << (t & 31u));
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------ summing the runs

constexpr int EG_THREADS = 128;
constexpr int EG_CHUNK = 64;   // pairs of a chunk, at most
constexpr int EG_AHEAD = 8;    // loads of a thread in flight (32768 tokens of 5120 bf16: 287 us, 298 with 4)
constexpr int EG_ZERO_ROWS = 8;

struct GradPlan {
  int chunk, n_chunks, tiles;
  unsigned run_blocks, zero_blocks;
  const uint2* pairs;
  const uint32_t* present;
  // [chunk][2][part_ld]: the sums of the run that comes from the chunk before, and of the one that goes on
  float* parts;
  long long part_ld;
  int join_tiles;
};

// The columns of a tile: EG_THREADS vectors.  `col0` is the tile's first one.
template <typename T, bool VEC>
__device__ __forceinline__ void write_grad(const EmbedArgs& a, uint32_t token, int col0, const float* sum) {
  using C = Cols<T, VEC>;
  T* row = static_cast<T*>(a.dst) + (long long)token * a.dst_ld + col0;
  float z[C::PER];
#pragma unroll
  for (int e = 0; e < C::PER; ++e) z[e] = sum[e] * a.scale;
  if (a.accumulate) {
    float old[C::PER];
    Elem<T>::unpack(C::load(row, threadIdx.x, 0, a.d - col0), old);
#pragma unroll
    for (int e = 0; e < C::PER; ++e) z[e] += old[e];
  }
  C::store(row, threadIdx.x, 0, a.d - col0, round_vec<T>(z));
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(EG_THREADS) k_embed_grad(EmbedArgs a, GradPlan p) {
  using C = Cols<T, VEC>;
  constexpr int PER = C::PER;
  __shared__ uint2 s_pair[EG_CHUNK + 2];  // the pair before the chunk, the chunk, the pair after it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.n_chunks > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel follows
  if (blockIdx.x >= p.run_blocks) {
    const long long v0 = (long long)(blockIdx.x - p.run_blocks) * EG_ZERO_ROWS;
    for (int r = 0; r < EG_ZERO_ROWS; ++r) {
      const long long v = v0 + r;
      if (v >= a.vocab) return;
      if ((__ldg(p.present + (v >> 5)) >> (v & 31)) & 1u) continue;
      T* row = static_cast<T*>(a.dst) + v * a.dst_ld;
      for (int col0 = 0; col0 < a.d; col0 += EG_THREADS * PER)
        C::store(row + col0, threadIdx.x, 0, a.d - col0, make_uint4(0u, 0u, 0u, 0u));
    }
    return;
  }
  const int c = blockIdx.x / p.tiles, tile = blockIdx.x - c * p.tiles;
  const int i0 = c * p.chunk, n = min(p.chunk, a.N - i0);
  const uint2 none = make_uint2(0xFFFFFFFFu, 0u);
  for (int i = threadIdx.x; i < n + 2; i += EG_THREADS) {
    const int g = i0 + i - 1;
    s_pair[i] = g >= 0 && g < a.N ? __ldg(p.pairs + g) : none;
  }
  __syncthreads();
  const int col0 = tile * EG_THREADS * PER;
  const T* grad = static_cast<const T*>(a.src) + col0;
  float sum[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) sum[e] = 0.f;
  bool from_before = s_pair[0].x == s_pair[1].x;
  for (int j = 0; j < n; j += EG_AHEAD) {
    uint4 x[EG_AHEAD];
#pragma unroll
    for (int q = 0; q < EG_AHEAD; ++q) {
      x[q] = make_uint4(0u, 0u, 0u, 0u);
      if (j + q < n && s_pair[j + q + 1].x < (uint32_t)a.vocab)
        x[q] = C::load(grad + (long long)s_pair[j + q + 1].y * a.src_ld, threadIdx.x, 0, a.d - col0);
    }
#pragma unroll
    for (int q = 0; q < EG_AHEAD; ++q) {
      if (j + q >= n) break;
      const uint32_t token = s_pair[j + q + 1].x;
      if (token >= (uint32_t)a.vocab) return;  // the padding, behind every token
      float z[PER];
      Elem<T>::unpack(x[q], z);
#pragma unroll
      for (int e = 0; e < PER; ++e) sum[e] += z[e];
      const bool goes_on = s_pair[j + q + 2].x == token;
      if (goes_on && j + q + 1 < n) continue;
      if (from_before || goes_on) {
        float* part = p.parts + ((long long)c * 2 + (from_before ? 0 : 1)) * p.part_ld + col0;
        if constexpr (VEC) {
#pragma unroll
          for (int e = 0; e < PER; e += 4)
            *reinterpret_cast<float4*>(part + threadIdx.x * PER + e) =
                make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < PER; ++e) part[C::col(threadIdx.x, 0, e)] = sum[e];
        }
      } else {
        write_grad<T, VEC>(a, token, col0, sum);
      }
      from_before = false;
#pragma unroll
      for (int e = 0; e < PER; ++e) sum[e] = 0.f;
    }
  }
}

// A run that starts in chunk c and goes on: the sum of its parts, for a tile of columns.  Warp w adds the parts w,
// w + 8, ..., and the warps' sums are added in order.
constexpr int EJ_WARPS = 8, EJ_VECS = 4, EJ_COLS = 128 * EJ_VECS;
template <typename T>
__global__ void __launch_bounds__(32 * EJ_WARPS) k_embed_join(EmbedArgs a, GradPlan p) {
  __shared__ float s_sum[EJ_WARPS][EJ_COLS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x / p.join_tiles, tile = blockIdx.x - c * p.join_tiles;
  const long long end = (long long)(c + 1) * p.chunk, start = end - p.chunk;
  if (end >= a.N) return;
  const uint32_t token = __ldg(p.pairs + end - 1).x, next = __ldg(p.pairs + end).x;
  const uint32_t prev = start > 0 ? __ldg(p.pairs + start - 1).x : 0xFFFFFFFFu;
  // no run goes on, or it comes from the chunk before
  if (token >= (uint32_t)a.vocab || next != token || (prev == token && __ldg(p.pairs + start).x == token)) return;
  // its last chunk: the last whose first pair has the token
  int last = c + 1;
  for (int k0 = c + 2;; k0 += 32) {
    const int k = k0 + lane;
    const bool same = k < p.n_chunks && __ldg(p.pairs + (long long)k * p.chunk).x == token;
    const uint32_t run = __ballot_sync(0xFFFFFFFFu, same);
    last += run == 0xFFFFFFFFu ? 32 : __ffs(~run) - 1;
    if (run != 0xFFFFFFFFu) break;
  }
  // part 0: of chunk c; part i: of chunk c + i
  const int n = last - c + 1;
  const float* from = p.parts + (long long)c * 2 * p.part_ld + tile * EJ_COLS + lane * 4;
  float4 sum[EJ_VECS];
#pragma unroll
  for (int v = 0; v < EJ_VECS; ++v) sum[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = warp; i < n; i += EJ_WARPS) {
#pragma unroll
    for (int v = 0; v < EJ_VECS; ++v) {
      const float4 x = *reinterpret_cast<const float4*>(from + (i == 0 ? 1 : 2LL * i) * p.part_ld + v * 128);
      sum[v].x += x.x;
      sum[v].y += x.y;
      sum[v].z += x.z;
      sum[v].w += x.w;
    }
  }
#pragma unroll
  for (int v = 0; v < EJ_VECS; ++v) *reinterpret_cast<float4*>(&s_sum[warp][v * 128 + lane * 4]) = sum[v];
  __syncthreads();
  for (int i = threadIdx.x; i < EJ_COLS; i += 32 * EJ_WARPS) {
    const int id = tile * EJ_COLS + i;
    if (id >= a.d) return;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < EJ_WARPS; ++w) t += s_sum[w][i];
    T* to = static_cast<T*>(a.dst) + (long long)token * a.dst_ld + id;
    t *= a.scale;
    if (a.accumulate) t += Elem<T>::to_f(*to);
    *to = Elem<T>::from_f(t);
  }
}

// Pairs per chunk: 64, fewer where that leaves the 152 SMs with less than two chunks each.  (The workspace goes by it,
// whose size is asked for without a device.)  1001 columns of fp32, with 64, 16 and 8 in a chunk: 2000 tokens 25, 17.1
// and 16.5 us, 5000 tokens 29, 20.2 and 22.6, 20011 tokens 40.5, 44 and 54.
int chunk_of(int N) { return N >= 64 * 304 ? 64 : N >= 16 * 304 ? 16 : 8; }

// Columns of a part, whole tiles of either type.
size_t part_width(int d) { return align_up((size_t)d, EG_THREADS * 8); }

struct GradLayout {
  size_t buf0, buf1, present, parts, total;
};
GradLayout grad_layout(int N, int vocab, int d) {
  GradLayout L;
  size_t off = WS_HEADER;
  L.buf0 = off;
  off = align_up(off + (size_t)N * 8, 256);
  L.buf1 = off;
  off = align_up(off + (size_t)N * 8, 256);
  L.present = off;
  off = align_up(off + ((size_t)vocab + 31) / 32 * 4, 256);
  L.parts = off;
  const int chunk = chunk_of(N);
  off = align_up(off + ((size_t)N + chunk - 1) / chunk * 2 * part_width(d) * 4, 256);
  L.total = off;
  return L;
}

template <typename T>
cudaError_t run_embed(const Ctx& c, const EmbedArgs& a) {
  constexpr int PER = Elem<T>::PER16;
  const bool vec = whole_vectors(a.src, a.src_ld, a.vocab, a.d, sizeof(T)) &&
                   whole_vectors(a.dst, a.dst_ld, a.N, a.d, sizeof(T));
  const unsigned units = vec ? (unsigned)(a.d / PER) : (unsigned)pieces(a.d, PER);
  const unsigned long long items = (unsigned long long)a.N * units;
  const bool few = items <= (unsigned long long)EM_THREADS * EM_VECS * EM_FEW * c.num_sms;
  const unsigned each = EM_THREADS * (few ? 1 : EM_VECS), grid = (unsigned)((items + each - 1) / each);
  return launch_pdl(c, "embed",
                    few ? (vec ? k_embed<T, true, 1> : k_embed<T, false, 1>)
                        : (vec ? k_embed<T, true, EM_VECS> : k_embed<T, false, EM_VECS>),
                    dim3(grid), dim3(EM_THREADS), 0, a, units);
}

// No tokens: rows of zeros.
template <typename T>
cudaError_t launch_zeros(const Ctx& c, const EmbedArgs& a) {
  return note_error(cudaMemset2DAsync(a.dst, (size_t)(a.vocab > 1 ? a.dst_ld : a.d) * sizeof(T), 0,
                                      (size_t)a.d * sizeof(T), (size_t)a.vocab, c.stream),
                    "cudaMemset2DAsync");
}

template <int BITS>
cudaError_t launch_sort(const Ctx& c, const EmbedArgs& a, int passes, uint2* const* buf, uint32_t* present) {
  static unsigned long long smem_done = 0;
  const cudaError_t e = allow_max_smem(k_token_sort<BITS>, c.device, &smem_done);
  if (e != cudaSuccess) return e;
  // one block for few tokens (gradients of 64 fp32 columns, 4096 rows: 1000 tokens 13.5 us, 15.3 by the cluster; 2000 tokens
  // 15.9 and 16.0; 4000 tokens 21.5 and 17.1)
  const unsigned ranks = a.N > TS_FEW ? TS_RANKS : 1;
  return launch_clusters(c, "token_sort", k_token_sort<BITS>, ranks, dim3(ranks), dim3(TS_THREADS),
                         (size_t)TS_WARPS * (1u << BITS) * 4, a.tokens, a.N, a.vocab, passes, buf[0], buf[1], present);
}

template <typename T>
cudaError_t run_embed_backward(const Ctx& c, const EmbedArgs& a) {
  constexpr int PER = Elem<T>::PER16;
  const GradLayout L = grad_layout(a.N, a.vocab, a.d);
  uint2* buf[2] = {reinterpret_cast<uint2*>(a.ws + L.buf0), reinterpret_cast<uint2*>(a.ws + L.buf1)};
  uint32_t* present = reinterpret_cast<uint32_t*>(a.ws + L.present);
  if (a.N == 0) return launch_zeros<T>(c, a);
  int key_bits = 0;
  while (a.vocab >> key_bits) ++key_bits;  // the largest key is vocab
  const int passes = (key_bits + TS_BITS - 1) / TS_BITS;
  const int bits = (key_bits + passes - 1) / passes;
  cudaError_t e = bits <= 6   ? launch_sort<6>(c, a, passes, buf, present)
                  : bits == 7 ? launch_sort<7>(c, a, passes, buf, present)
                  : bits == 8 ? launch_sort<8>(c, a, passes, buf, present)
                              : launch_sort<TS_BITS>(c, a, passes, buf, present);
  if (e != cudaSuccess) return e;
  const bool vec = whole_vectors(a.src, a.src_ld, a.N, a.d, sizeof(T)) &&
                   whole_vectors(a.dst, a.dst_ld, a.vocab, a.d, sizeof(T));
  GradPlan p = {};
  p.chunk = chunk_of(a.N);
  p.n_chunks = (int)(((long long)a.N + p.chunk - 1) / p.chunk);
  p.tiles = (a.d + EG_THREADS * PER - 1) / (EG_THREADS * PER);
  p.run_blocks = (unsigned)p.n_chunks * (unsigned)p.tiles;
  p.zero_blocks = a.accumulate ? 0u : (unsigned)((a.vocab + EG_ZERO_ROWS - 1) / EG_ZERO_ROWS);
  p.pairs = buf[(passes - 1) & 1];
  p.present = present;
  p.parts = reinterpret_cast<float*>(a.ws + L.parts);
  p.part_ld = (long long)part_width(a.d);
  p.join_tiles = (a.d + EJ_COLS - 1) / EJ_COLS;
  e = launch_pdl(c, "embed_grad", vec ? k_embed_grad<T, true> : k_embed_grad<T, false>,
                 dim3(p.run_blocks + p.zero_blocks), dim3(EG_THREADS), 0, a, p);
  if (e != cudaSuccess || p.n_chunks == 1) return e;
  return launch_pdl(c, "embed_join", k_embed_join<T>, dim3((unsigned)p.n_chunks * (unsigned)p.join_tiles),
                    dim3(32 * EJ_WARPS), 0, a, p);
}

}  // namespace

size_t embed_backward_workspace(int N, int vocab, int d, int) { return grad_layout(N, vocab, d).total; }

cudaError_t launch_embed(const Ctx& c, const EmbedArgs& a, int dtype) {
  return dtype == DH_BF16 ? run_embed<__nv_bfloat16>(c, a) : run_embed<float>(c, a);
}
cudaError_t launch_embed_backward(const Ctx& c, const EmbedArgs& a, int dtype) {
  return dtype == DH_BF16 ? run_embed_backward<__nv_bfloat16>(c, a) : run_embed_backward<float>(c, a);
}

}  // namespace dh
