// One step of beam search: the M best of score[w] + z[w, v]/T - log sum exp(z[w, :]/T) over a
// request's beams w and the vocabulary v (definition at dh_beam_select in dh.h).
//
// The pass over the logits (row_stats.cu, the step's traffic: HBM-bound) leaves a (max, sum) pair
// per segment of a row.  k_beam_pick then works from those pairs, one block per request:
//   1. each beam's normaliser, hence base[w] = score[w] - log sum exp((z - max)/T), in 64 bits: two
//      candidates of different beams are ordered by it, so its error (about 1e-7, from the sums' fp32
//      exponentials) decides which of two near ones comes first;
//   2. a bound: every thread's best segment maximum is the score of some candidate, so the M-th
//      largest of them is one that at least M candidates reach.  It only has to be a lower bound, so
//      it is taken in fp32, each score lowered by more than its rounding;
//   3. the segments whose maximum reaches the bound are read again (about M of them, from L2), and
//      the elements that reach it become candidates with their scores in 64 bits;
//   4. candidates are ranked by (score desc, beam asc, token asc), a strict order, so the result
//      does not depend on the order in which they were found.
// Where so many elements are level with the bound that the list overflows (rows of few distinct
// values), the segments are walked in order instead, keeping the M best so far; a later segment
// then enters only with a score above the M-th best (equal ones come behind it in the order), so
// even constant rows end after the first segments.
//
// k_beam_pick is a chain of latencies (128 requests of 16 beams, M = 16: 8 us, of it the combination
// 1.4, logarithms 0.5, bound 1.5, search of the segments 0.5, elements read again 2, scores and order 2).
// What runs once is kept out of line: unrolled code has to come from memory first.
//
// The bound needs M maxima of live beams (for M up to 64: M of the 128 groups of four threads).  Where the
// rest of a request's beams is unused, finished or broken there may be fewer, with one ended beam already
// where all segments together are hardly more than 4 M; the bound then asks nothing and the walk takes
// over, whose every segment costs a selection of its own.  A step of one live beam among
// W, against all of them live: 8 x 32000 bf16, M = 16: 519 us / 12; 8 requests of 16 x 50257 fp32, M = 32:
// 1363 / 23; of 16 x 151936 bf16, M = 200: 3206 / 62, M = 16 (149 segments are enough): 13 / 19.  One of 16
// beams of 4096 fp32 logits ended, M = 32: 1448 / 21.
#include <cstddef>

#include "rows.cuh"

namespace dh {
namespace {

constexpr int BP_THREADS = 512;
constexpr int BP_WARPS = BP_THREADS / 32;
constexpr int BP_CAP = 2048;      // candidates held at once (at least DH_MAX_BEAM_OUT + one segment)
constexpr int BP_SEGS = 1024;     // segments held at once
constexpr int BP_BATCH = 10;      // vectors of a warp in flight
// Segments of a thread in registers and segment maxima in shared memory, both for 16 beams of 152K bf16
// logits; what is beyond them is read again from L2, which costs next to nothing (32 requests of such
// beams: 34.6 us, with nothing staged 34.7; in fp32 they leave both).
constexpr int BP_HELD = 5;
constexpr int BP_STAGE = 2560;

// Order-preserving map of a double onto uint64 (-0 is folded onto +0).
__device__ __forceinline__ unsigned long long dkey(double x) {
  const long long b = __double_as_longlong(x + 0.0);
  return b < 0 ? ~(unsigned long long)b : ((unsigned long long)b | 0x8000000000000000ull);
}
__device__ __forceinline__ double dkey_inv(unsigned long long k) {
  return __longlong_as_double((k >> 63) ? (long long)(k & 0x7FFFFFFFFFFFFFFFull) : (long long)~k);
}

struct BeamArgs {
  const void* logits;
  long long rs, ws;  // strides of a request's and a beam's row, in elements
  const float* score;
  const int32_t* finished;
  const float2* seg;
  int W, vocab, M, n_seg, pad_token;
  float temperature, inv_t;
  double inv_t64;
  int32_t* parent;
  int32_t* token;
  float* score_out;
};

struct BeamSmem {
  alignas(16) unsigned long long key[BP_CAP];
  uint32_t pos[BP_CAP];
  double base[DH_MAX_BEAMS];   // score of the row's largest logit; -inf: no candidates of its own
  float base32[DH_MAX_BEAMS];
  float top[DH_MAX_BEAMS];     // the row's largest logit
  float sum_hi[DH_MAX_BEAMS], sum_lo[DH_MAX_BEAMS], score[DH_MAX_BEAMS];
  bool done[DH_MAX_BEAMS];     // finished, with a score
  float zthr[DH_MAX_BEAMS];    // logits from here on reach the bound
  float seg_max[BP_STAGE];
  float tau;
  uint32_t segs[BP_SEGS];
  int count[2][BP_WARPS];
  unsigned long long last_key;
  uint32_t last_pos;
  int n, n_segs, next;
};
// the keys' place is read 16 bytes at a time before they stand there (k_beam_pick, part 2)
static_assert(alignof(BeamSmem) % 16 == 0 && offsetof(BeamSmem, key) % 16 == 0, "16-byte loads from BeamSmem::key");

// Sum of x over the block.  `turn` alternates between calls, so one barrier per call is enough.
__device__ __forceinline__ int block_count(BeamSmem& s, int x, int& turn) {
  const int c = __reduce_add_sync(0xFFFFFFFFu, x);
  if ((threadIdx.x & 31) == 0) s.count[turn][threadIdx.x >> 5] = c;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < BP_WARPS; ++w) total += s.count[turn][w];
  turn ^= 1;
  return total;
}

// A lower bound of the exact score b + (z - top)/T from its fp32 terms: their roundings are together
// below 2^-22 of each term.
__device__ __forceinline__ float score_below(float b, float top, float z, float inv_t) {
  const float x = (z - top) * inv_t, s = b + x;
  return s - (fabsf(b) + fabsf(x) + fabsf(s)) * 2.384185791015625e-7f;
}

// The score of logit z of beam w, in 64 bits.
__device__ __forceinline__ double exact_score(const BeamSmem& s, const BeamArgs& a, int w, float z) {
  return s.base[w] + ((double)z - (double)s.top[w]) * a.inv_t64;
}

// The bound's lowest logit per beam: z >= zthr[w] for every z whose score is tau or more.  The
// slack is far above the rounding of the terms (2^-24 each).
__device__ __forceinline__ void set_thresholds(BeamSmem& s, const BeamArgs& a, float tau) {
  for (int w = threadIdx.x; w < a.W; w += BP_THREADS) {
    const float b = s.base32[w];
    const float top = s.top[w];
    const float slack = ((fabsf(tau) + fabsf(b)) * a.temperature + fabsf(top)) * 9.5367431640625e-7f + 1e-30f;
    const float z = top + (tau - b) * a.temperature - slack;
    // terms that overflow set no bound
    s.zthr[w] = b == -INFINITY ? INFINITY : (z == z && z < INFINITY ? z : -INFINITY);
  }
}

// Leaves the best M of the list's s.n > M candidates in its first M places (in no order): the M-th
// key by descent over its bits with block-wide counts, then, among equal keys, the M-th position.
__device__ __noinline__ void keep_best(BeamSmem& s, int M) {
  constexpr int PER = BP_CAP / BP_THREADS;
  unsigned long long k[PER];
  uint32_t p[PER];
  const int n = s.n;
  int turn = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = threadIdx.x + i * BP_THREADS;
    k[i] = j < n ? s.key[j] : 0ull;  // below every key of a number
    p[i] = j < n ? s.pos[j] : 0xFFFFFFFFu;
  }
  unsigned long long t = 0;
  for (int b = 63; b >= 0; --b) {
    const unsigned long long u = t | (1ull << b);
    int c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += k[i] >= u;
    if (block_count(s, c, turn) >= M) t = u;
  }
  int above = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) above += k[i] > t;
  above = block_count(s, above, turn);
  // of the keys equal to t the lowest M - above positions: the largest bound q with fewer than that
  // many positions below it
  const int room = M - above;
  uint32_t q = 0;
  for (int b = 31; b >= 0; --b) {
    const uint32_t u = q | (1u << b);
    int c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += k[i] == t && p[i] < u;
    if (block_count(s, c, turn) < room) q = u;
  }
  __syncthreads();
  if (threadIdx.x == 0) s.n = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = threadIdx.x + i * BP_THREADS;
    if (j < n && (k[i] > t || (k[i] == t && p[i] <= q))) {
      const int at = atomicAdd(&s.n, 1);
      s.key[at] = k[i];
      s.pos[at] = p[i];
    }
  }
  __syncthreads();
}

// Adds the elements of vector u (ids id ..) of beam w that reach the bound.  Their logits stand where
// the keys will (score_pushed).
template <typename T>
__device__ __noinline__ void push_elems(BeamSmem& s, const BeamArgs& a, uint4 u, int id, int w, float zthr) {
  constexpr int PER = Elem<T>::PER16;
  float z[PER];
  Elem<T>::unpack(u, z);
#pragma unroll
  for (int e = 0; e < PER; ++e)
    if (z[e] >= zthr && z[e] > -INFINITY) {
      const int at = atomicAdd(&s.n, 1);
      if (at < BP_CAP) {
        s.key[at] = __float_as_uint(z[e]);
        s.pos[at] = (uint32_t)w * (uint32_t)a.vocab + (uint32_t)(id + e);
      }
    }
}
template <typename T>
__device__ __forceinline__ void push_vec(BeamSmem& s, const BeamArgs& a, const uint4& u, int id, int w, float zthr) {
  const uint4 one[1] = {u};
  if (vec_max<T>(one) >= zthr) push_elems<T>(s, a, u, id, w, zthr);  // few vectors
}

// The keys of the candidates from number `first` on, whose logits were pushed.
__device__ __noinline__ void score_pushed(BeamSmem& s, const BeamArgs& a, int first) {
  for (int i = first + (int)threadIdx.x; i < s.n; i += BP_THREADS)
    s.key[i] = dkey(exact_score(s, a, (int)(s.pos[i] / (uint32_t)a.vocab), __uint_as_float((uint32_t)s.key[i])));
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(BP_THREADS) k_beam_pick(BeamArgs a) {
  constexpr int PER = Elem<T>::PER16;
  constexpr int SEG = row_seg<T>();
  __shared__ BeamSmem s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = a.W, M = a.M, n_seg = a.n_seg, n_all = W * n_seg;
  const size_t row0 = (size_t)blockIdx.x * W;
  const T* rows = static_cast<const T*>(a.logits) + (long long)blockIdx.x * a.rs;
  const float2* seg = a.seg + row0 * n_seg;
  const float* score = a.score + row0;
  const int32_t* finished = a.finished ? a.finished + row0 : nullptr;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // 1. the beams: a warp each for the sums, then a lane each for the logarithms (64-bit operations take
  // a warp 16 cycles whatever its active lanes, so they are done 32 at a time)
  if (tid == 0) s.n = s.n_segs = 0;
  const bool staged = n_all <= BP_STAGE;  // the segments' maxima fit shared memory
  for (int w = warp; w < W; w += BP_WARPS) {
    const float sc = __ldg(score + w);
    const bool fin = finished && __ldg(finished + w) != 0;
    const bool live = fabsf(sc) < INFINITY && !fin;
    // a beam that is not live has no pairs; what stands in their place is combined all the same, so
    // that no load waits for another, and not used
    float m;
    Sum2 sum;
    row_combine(seg + (size_t)w * n_seg, n_seg, a.inv_t, &m, &sum, staged ? &s.seg_max[w * n_seg] : nullptr);
    const float total = sum.hi, rest = sum.lo;
    if (lane == 0) {
      // a row of -inf, and one with a NaN or +inf, has no distribution
      const bool good = live && fabsf(m) < INFINITY && total + rest < INFINITY;
      s.top[w] = good ? m : 0.f;
      s.sum_hi[w] = good ? total : 0.f;  // 0: no candidates of its own
      s.sum_lo[w] = rest;
      s.score[w] = sc;
      s.done[w] = fin && fabsf(sc) < INFINITY;
    }
  }
  __syncthreads();
  for (int w = tid; w < W; w += BP_THREADS) {
    double b = -(double)INFINITY;
    if (s.sum_hi[w] > 0.f) {
      const Sum2 l = log_sum(s.sum_hi[w], s.sum_lo[w]);
      b = ((double)s.score[w] - (double)l.hi) - (double)l.lo;
    }
    s.base[w] = b;
    s.base32[w] = (float)b;
  }
  __syncthreads();
  auto seg_max = [&](int i) { return staged ? s.seg_max[i] : seg[i].x; };
  // i / n_seg for i < W n_seg: (i + 0.5) / n_seg is at least 0.5 / n_seg >= 2^-13 away from an integer
  // (n_seg <= 4096), the error of the product below 128 x 1.5 x 2^-23 < 2^-15
  const float inv_seg = 1.f / (float)n_seg;
  auto beam_of = [&](int i) { return __float2int_rz(((float)i + 0.5f) * inv_seg); };

  // 2. the bound.  Few segments: the threads' best elements instead of their best segments
  const bool by_elem = n_all < 4 * M;
  float best = -INFINITY;
  // a thread's first segments stay in registers: beam and maximum (-inf: not to be looked at)
  int held_w[BP_HELD] = {};
  float held_m[BP_HELD];
#pragma unroll
  for (int q = 0; q < BP_HELD; ++q) held_m[q] = -INFINITY;
  if (by_elem) {
    for (int i = warp; i < n_all; i += BP_WARPS) {
      const int w = i / n_seg, id0 = (i - w * n_seg) * SEG + lane * PER;
      if (s.base32[w] == -INFINITY) continue;
      uint4 u[ROW_SEG_VECS];
#pragma unroll
      for (int v = 0; v < ROW_SEG_VECS; ++v)
        u[v] = row_vec<T, ALIGNED, true>(rows + w * a.ws, id0 + v * 32 * PER, a.vocab);
      best = fmaxf(best, score_below(s.base32[w], s.top[w], vec_max<T>(u), a.inv_t));
    }
  } else {
#pragma unroll
    for (int q = 0; q < BP_HELD; ++q) {
      const int i = tid + q * BP_THREADS;
      if (i >= n_all) break;
      const int w = beam_of(i);
      if (s.base32[w] == -INFINITY) continue;
      held_w[q] = w;
      held_m[q] = seg_max(i);
      best = fmaxf(best, score_below(s.base32[w], s.top[w], held_m[q], a.inv_t));
    }
    for (int i = tid + BP_HELD * BP_THREADS; i < n_all; i += BP_THREADS) {
      const int w = beam_of(i);
      if (s.base32[w] != -INFINITY) best = fmaxf(best, score_below(s.base32[w], s.top[w], seg_max(i), a.inv_t));
    }
  }
  if (finished)
    for (int w = tid; w < W; w += BP_THREADS)
      if (s.done[w]) best = fmaxf(best, s.score[w]);
  // The M-th largest: for up to 64 by the ranks of 128 maxima of four threads each (a few more
  // candidates reach it: 37 where 32 are asked for), else by descent over the leading bits of the
  // threads' maxima, with a block-wide count each (19 barriers; 32 requests of 16 beams, M = 16: 34.8 us
  // against 34.6; 8 of fp32 rows 23.3 against 23.8).
  float tau;
  if (M <= 64) {
    best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, 1));
    best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, 2));
    float* const four = reinterpret_cast<float*>(s.key);  // [128], not yet in use
    if ((lane & 3) == 0) four[tid >> 2] = best;
    __syncthreads();
    // maximum tid / 4 against a quarter of them per lane
    const int me = tid >> 2;
    const float mine = four[me];
    int rank = 0;
#pragma unroll
    for (int q = 0; q < BP_THREADS / 64; ++q) {
      const int j = q * 16 + (tid & 3) * 4;
      const float4 o = *reinterpret_cast<const float4*>(four + j);
      rank += (o.x > mine || (o.x == mine && j < me)) + (o.y > mine || (o.y == mine && j + 1 < me)) +
              (o.z > mine || (o.z == mine && j + 2 < me)) + (o.w > mine || (o.w == mine && j + 3 < me));
    }
    rank += __shfl_xor_sync(0xFFFFFFFFu, rank, 1);
    rank += __shfl_xor_sync(0xFFFFFFFFu, rank, 2);
    if ((lane & 3) == 0 && rank == M - 1) s.tau = mine;  // ranks are distinct
    __syncthreads();
    tau = s.tau;
  } else {
    const uint32_t mine = fkey(best);
    uint32_t t = 0;
    for (int b = 31; b >= 13; --b) {
      const uint32_t u = t | (1u << b);
      if (__syncthreads_count(mine >= u) >= M) t = u;
    }
    tau = t == 0 ? -INFINITY : fkey_inv(t);
  }
  if (!(tau > -INFINITY && tau < INFINITY)) tau = -INFINITY;  // a bound that no number has asks nothing
  set_thresholds(s, a, tau);
  __syncthreads();

  // 3. the segments and elements that reach it
  auto reach = [&](int i, int w, float m) {
    if (m >= s.zthr[w] && m > -INFINITY) {
      const int at = atomicAdd(&s.n_segs, 1);
      if (at < BP_SEGS) s.segs[at] = (uint32_t)i;
    }
  };
  if (!by_elem) {
#pragma unroll
    for (int q = 0; q < BP_HELD; ++q)
      if (held_m[q] != -INFINITY) reach(tid + q * BP_THREADS, held_w[q], held_m[q]);
  }
  for (int i = tid + (by_elem ? 0 : BP_HELD * BP_THREADS); i < n_all; i += BP_THREADS) {
    const int w = beam_of(i);
    if (s.base32[w] != -INFINITY) reach(i, w, seg_max(i));
  }
  if (finished)
    for (int w = tid; w < W; w += BP_THREADS)
      if (s.done[w]) {
        const int at = atomicAdd(&s.n, 1);
        s.pos[at] = (uint32_t)w * (uint32_t)a.vocab;
        s.key[at] = dkey((double)s.score[w]);
      }
  __syncthreads();
  const int n_fin = s.n;  // a finished beam's candidate each (W <= DH_MAX_BEAMS: they fit)
  const bool many = s.n_segs > BP_SEGS;
  __syncthreads();
  if (!many) {
    // a warp's vectors BP_BATCH at a time, so that up to 40 segments take one trip to memory
    const int n_rows = s.n_segs * ROW_SEG_VECS;
    for (int i0 = warp; i0 < n_rows; i0 += BP_WARPS * BP_BATCH) {
      uint4 u[BP_BATCH];
#pragma unroll
      for (int q = 0; q < BP_BATCH; ++q) {
        const int i = i0 + q * BP_WARPS;
        if (i >= n_rows) continue;
        const int sg = (int)s.segs[i / ROW_SEG_VECS], w = beam_of(sg);
        u[q] = row_vec<T, ALIGNED, true>(rows + w * a.ws,
                                   (sg - w * n_seg) * SEG + (i % ROW_SEG_VECS * 32 + lane) * PER, a.vocab);
      }
#pragma unroll
      for (int q = 0; q < BP_BATCH; ++q) {
        const int i = i0 + q * BP_WARPS;
        if (i >= n_rows) continue;
        const int sg = (int)s.segs[i / ROW_SEG_VECS], w = beam_of(sg);
        push_vec<T>(s, a, u[q], (sg - w * n_seg) * SEG + (i % ROW_SEG_VECS * 32 + lane) * PER, w, s.zthr[w]);
      }
    }
  }
  __syncthreads();
  if (!many && s.n <= BP_CAP) {
    score_pushed(s, a, n_fin);
    __syncthreads();
    if (s.n > 256 && s.n > M) keep_best(s, M);  // ranking below compares all pairs
  } else {
    // too many level with the bound: walk the segments in (beam, token) order, keeping the M best.
    // Once M are held a segment enters only if its maximum at its first id would rank before the
    // M-th best (a finished beam's candidate may be held ahead of its turn).
    __syncthreads();
    if (tid == 0) s.n = n_fin;  // the finished beams' candidates are the list's first
    __syncthreads();
    if (s.n > M) keep_best(s, M);
    int at = 0;
    for (;;) {
      // the M-th best pair, once M are held (s.n == M then)
      unsigned long long last = 0;
      uint32_t last_pos = 0xFFFFFFFFu;
      const int held = s.n;
      if (held >= M) {
        __syncthreads();
        if (tid == 0) {
          s.last_key = ~0ull;
          s.last_pos = 0;
        }
        __syncthreads();
        if (tid < M) atomicMin(&s.last_key, s.key[tid]);
        __syncthreads();
        last = s.last_key;
        if (tid < M && s.key[tid] == last) atomicMax(&s.last_pos, s.pos[tid]);
        __syncthreads();
        last_pos = s.last_pos;
      }
      // the next segment that can hold a better one: BP_THREADS looked at a time
      int found = n_all;
      for (int i0 = at; i0 < n_all; i0 += BP_THREADS) {
        const int i = i0 + tid;
        bool ok = false;
        if (i < n_all) {
          const int w = i / n_seg;
          if (s.base32[w] != -INFINITY) {
            const float m = seg_max(i);
            if (m > -INFINITY && m >= s.zthr[w]) {
              const unsigned long long k = dkey(exact_score(s, a, w, m));
              ok = k > last ||
                   (k == last && (uint32_t)w * (uint32_t)a.vocab + (uint32_t)((i - w * n_seg) * SEG) < last_pos);
            }
          }
        }
        if (tid == 0) s.next = n_all;
        __syncthreads();
        if (ok) atomicMin(&s.next, i);
        __syncthreads();
        found = s.next;
        __syncthreads();
        if (found < n_all) break;
      }
      if (found >= n_all) break;
      const int w = found / n_seg, id0 = (found - w * n_seg) * SEG;
      if (warp < ROW_SEG_VECS) {
        const int id = id0 + (warp * 32 + lane) * PER;
        const uint4 u = row_vec<T, ALIGNED, true>(rows + w * a.ws, id, a.vocab);
        push_vec<T>(s, a, u, id, w, s.zthr[w]);
      }
      __syncthreads();
      score_pushed(s, a, held);
      __syncthreads();
      if (s.n > M) keep_best(s, M);
      at = found + 1;
    }
  }
  __syncthreads();

  // 4. the order
  const int n = s.n;
  int32_t* parent = a.parent + (size_t)blockIdx.x * M;
  int32_t* token = a.token + (size_t)blockIdx.x * M;
  float* out = a.score_out + (size_t)blockIdx.x * M;
  // a candidate's rank is the number that come before it, counted by eight lanes
  for (int i0 = 0; i0 < n; i0 += BP_THREADS / 8) {
    const int i = i0 + (tid >> 3), at = min(i, n - 1);
    const unsigned long long k = s.key[at];
    const uint32_t p = s.pos[at];
    int rank = 0;
    for (int j = tid & 7; j < n; j += 8) rank += s.key[j] > k || (s.key[j] == k && s.pos[j] < p);
    rank += __shfl_xor_sync(0xFFFFFFFFu, rank, 1);
    rank += __shfl_xor_sync(0xFFFFFFFFu, rank, 2);
    rank += __shfl_xor_sync(0xFFFFFFFFu, rank, 4);
    if (i < n && rank < M && (tid & 7) == 0) {
      const int w = (int)(p / (uint32_t)a.vocab);
      parent[rank] = w;
      token[rank] = s.done[w] ? a.pad_token : (int)(p - (uint32_t)w * (uint32_t)a.vocab);
      out[rank] = (float)dkey_inv(k);
    }
  }
  for (int i = n + tid; i < M; i += BP_THREADS) {
    parent[i] = token[i] = -1;
    out[i] = -INFINITY;
  }
}

template <typename T>
cudaError_t run(const Ctx& c, const BeamArgs& a, int R) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)R);
  cfg.blockDim = dim3(BP_THREADS);
  cfg.stream = c.stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const bool aligned = rows_aligned(a.logits, a.rs, a.ws, R, a.W, (int)sizeof(T));
  prof_before("beam_pick", c.stream);
  const cudaError_t e = aligned ? cudaLaunchKernelEx(&cfg, k_beam_pick<T, true>, a)
                                : cudaLaunchKernelEx(&cfg, k_beam_pick<T, false>, a);
  prof_after(c.stream);
  return e;
}

}  // namespace

cudaError_t launch_beam_select(const Ctx& c, const void* logits, long long rs, long long ws, const float* score,
                               const int32_t* finished, const float2* seg, int R, int W, int vocab, int M, int dtype,
                               float temperature, int pad_token, int32_t* parent, int32_t* token, float* score_out) {
  BeamArgs a{logits, rs, ws, score, finished, seg, W, vocab, M, row_segments(vocab, dtype), pad_token, temperature,
             1.f / temperature, 1.0 / (double)temperature, parent, token, score_out};
  return dtype == DH_BF16 ? run<__nv_bfloat16>(c, a, R) : run<float>(c, a, R);
}

}  // namespace dh
