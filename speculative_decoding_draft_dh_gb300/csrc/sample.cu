// Sampling one token per row of logits with temperature, top-k, top-p and min-p from a given uniform (definition
// at dh_sample in dh.h).
//
// In the order of a row's tokens by (logit desc, id asc) every filter keeps a prefix, and the drawn token is the
// one at which the prefix's running sum of weights passes u times its mass.  So everything is a search for a
// place in that order: by count (top-k) or by mass (top-p, the draw).  A search descends over the order-preserving
// keys of the logits: a histogram of at most 2048 bins over a range of keys (counts and masses), the bin that holds
// the place, then that bin's keys, until one key is left; tokens of one key have one weight, so the place among
// them is a division, and their order is that of the ids.
//
// Which token a uniform falls on hangs on the running sums, so the weights exp((z - max)/T) are integers: fixed
// point with S fraction bits relative to a power of two near the largest, S = 62 - log2(vocab), so that a row's
// masses fit 64 bits.  Their sums are exact, whatever the order of the atomics.  2^(z c), c = log2(e)/T, is taken as
// 2^(k/64) 2^r with k the rounded 64 z c: 2^(k/64) from a table, exact to 2^-29, and 2^r - 1, |r| < 2^-7 + 2^-9,
// by a cubic in fp32 whose rounding is below 2^-29 of the weight; c in two floats, so that z c is exact to 2^-31.
#include "layers.cuh"
#include "rows.cuh"

namespace dh {
namespace {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_BINS = 2048;

using u64 = unsigned long long;

// ------------------------------------------------------------------ weights

// 2^(j/64): as an integer with 28 fraction bits, and as that value in fp32.
struct ExpTable {
  uint32_t q[64];
  float f[64];
};
constexpr ExpTable make_table() {
  ExpTable t = {};
  for (int j = 0; j < 64; ++j) {
    double x = j * (0.693147180559945309417 / 64), term = 1, sum = 1;
    for (int n = 1; n < 20; ++n) {
      term *= x / n;
      sum += term;
    }
    sum *= 268435456.0;
    t.q[j] = (uint32_t)(sum + 0.5);
    t.f[j] = (float)sum;
  }
  return t;
}
__device__ const ExpTable g_exp_table = make_table();

constexpr float EXP_MAGIC = 196608.f;  // 1.5 2^17: adding it rounds to multiples of 1/64
constexpr int EXP_MAGIC_BITS = 0x48400000;

// The weights of a row whose largest logit is m at temperature t.  z c has to stay below 2^15 for the fp32 form;
// beyond that (huge logits, tiny temperatures) `far` takes 64-bit arithmetic.
struct Weights {
  float ch, cl, zlow;
  int e_ref, frac;  // the largest weight is in [2^frac, 2^(frac + 1)]
  bool far;
  double m, c;
  const ExpTable* tab;  // in shared memory
  __device__ Weights(float m_, float t, int frac_, const ExpTable* tab_) : frac(frac_), m(m_), tab(tab_) {
    c = 1.4426950408889634 / (double)t;
    ch = (float)c;
    cl = (float)(c - (double)ch);
    far = !(fabs(m * c) < 32000.0 && c < 1e38);
    const double low = m - (frac + 2) / c;  // weights below 2^-(frac + 1)
    zlow = low < -3.4e38 ? -3.4028234e38f : (float)low;
    e_ref = 0;
    if (!far) e_ref = (__float_as_int(fmaf(m_, ch, EXP_MAGIC)) - EXP_MAGIC_BITS) >> 6;
  }
  __device__ __forceinline__ u64 operator()(float z) const {
    if (!(z >= zlow)) return 0;
    uint32_t q;
    int down;
    if (__builtin_expect(far, 0)) {
      const double x = ((double)z - m) * c, e = floor(x);
      if (!(e > -64.0)) return 0;
      q = (uint32_t)rint(exp2(x - e) * 268435456.0);
      down = -(int)e;
    } else {
      const float k = fmaf(z, ch, EXP_MAGIC), kf = k - EXP_MAGIC;
      const float r = fmaf(z, cl, fmaf(z, ch, -kf));
      const int ki = __float_as_int(k) - EXP_MAGIC_BITS, j = ki & 63;
      // 2^r - 1 by its series
      const float x = r * fmaf(r, fmaf(r, 0.0555041087f, 0.240226507f), 0.693147181f);
      // added to 1.5 2^23, which rounds to an integer in the low bits; |tab.f x| < 2^22
      q = tab->q[j] + (uint32_t)(__float_as_int(fmaf(tab->f[j], x, 12582912.f)) - 0x4B400000);
      down = min(e_ref - (ki >> 6), 63);
    }
    return ((u64)q << (frac - 28)) >> down;
  }
};

// Order-preserving keys: of fp32 logits 32 bits, of bf16 logits 16.
template <typename T>
__device__ __forceinline__ uint32_t key_of(float z) {
  return sizeof(T) == 4 ? fkey(z) : fkey(z) >> 16;
}
// The smallest key of T whose value is at least x.
template <typename T>
__device__ __forceinline__ uint32_t key_at_least(float x) {
  const uint32_t k = fkey(x);
  if (sizeof(T) == 4) return k;
  // a negative bf16 value's key has ones where the fp32 key goes on, a positive one's zeros
  return (k & 0x80000000u) ? (k + 0xFFFFu) >> 16 : k >> 16;
}

// ------------------------------------------------------------------ the search

struct SampleSmem {
  u64 mass[SP_BINS];
  uint32_t count[SP_BINS];
  ExpTable tab;
  u64 warp_mass[SP_WARPS];
  uint32_t warp_count[SP_WARPS];
  float warp_max[SP_WARPS];
  int bin, last;
  u64 bin_mass, above_mass;
  uint32_t bin_count, above_count;
};

// A place in the order: all tokens above `key`, of which there are `above` with mass `above_mass`, and the tokens
// of that key: n_equal, each of weight w.
struct Place {
  uint32_t key, above, n_equal;
  u64 above_mass, w;
};

// f(value, id) of every logit of the row.
template <typename T, bool ALIGNED, typename F>
__device__ __forceinline__ void each(const T* row, int vocab, F f) {
  constexpr int PER = Elem<T>::PER16;
  for (int id = threadIdx.x * PER; id < vocab; id += SP_THREADS * PER) {
    float x[PER];
    Elem<T>::unpack(row_vec<T, ALIGNED>(row, id, vocab), x);
#pragma unroll
    for (int e = 0; e < PER; ++e) f(x[e]);
  }
}

// The first place with `want` tokens or more (BY_COUNT), or with a mass of want or more (STRICT: more than want),
// among the keys [lo, hi]; the last place where there is none.  hi is the row's largest key.
template <typename T, bool ALIGNED, bool BY_COUNT, bool STRICT>
__device__ __noinline__ Place descend(SampleSmem& s, const T* row, int vocab, uint32_t lo, uint32_t hi, u64 want,
                                      const Weights& weight) {
  u64 above_mass = 0;
  uint32_t above = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (;;) {
    const int bits = 32 - __clz(hi - lo), sh = bits > 11 ? bits - 11 : 0;
    for (int b = threadIdx.x; b < SP_BINS; b += SP_THREADS) {
      s.mass[b] = 0;
      s.count[b] = 0;
    }
    if (threadIdx.x == 0) s.bin = s.last = -1;
    __syncthreads();
    each<T, ALIGNED>(row, vocab, [&](float z) {
      const uint32_t k = key_of<T>(z);
      if (k >= lo && k <= hi) {
        const uint32_t b = (hi - k) >> sh;
        atomicAdd(&s.count[b], 1u);
        const u64 w = weight(z);
        if (w) atomicAdd(&s.mass[b], w);
      }
    });
    __syncthreads();
    // inclusive sums over the bins, four to a thread
    constexpr int OWN = SP_BINS / SP_THREADS;
    u64 m = 0;
    uint32_t c = 0;
    const int b0 = threadIdx.x * OWN;
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
      m += s.mass[b0 + q];
      c += s.count[b0 + q];
    }
    u64 mi = m;
    uint32_t ci = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 x = __shfl_up_sync(0xFFFFFFFFu, mi, o);
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, ci, o);
      if (lane >= o) {
        mi += x;
        ci += y;
      }
    }
    if (lane == 31) {
      s.warp_mass[warp] = mi;
      s.warp_count[warp] = ci;
    }
    __syncthreads();
    u64 ma = above_mass + mi - m;
    uint32_t ca = above + ci - c;
    for (int w = 0; w < warp; ++w) {
      ma += s.warp_mass[w];
      ca += s.warp_count[w];
    }
    auto reached = [&](u64 mass, uint32_t count) {
      return BY_COUNT ? count >= want : STRICT ? mass > want : mass >= want;
    };
    int last = -1;
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
      const u64 mb = s.mass[b0 + q];
      const uint32_t cb = s.count[b0 + q];
      if (cb) last = b0 + q;
      if (!reached(ma, ca) && reached(ma + mb, ca + cb)) {
        s.bin = b0 + q;
        s.bin_mass = mb;
        s.bin_count = cb;
        s.above_mass = ma;
        s.above_count = ca;
      }
      ma += mb;
      ca += cb;
    }
    if (last >= 0) atomicMax(&s.last, last);
    __syncthreads();
    if (s.bin < 0) {
      // the sums never reach it: the last bin that holds a token
      if (s.last >= b0 && s.last < b0 + OWN) {
        for (int q = OWN - 1; b0 + q > s.last; --q) {
          ma -= s.mass[b0 + q];
          ca -= s.count[b0 + q];
        }
        s.bin_mass = s.mass[s.last];
        s.bin_count = s.count[s.last];
        s.above_mass = ma - s.bin_mass;
        s.above_count = ca - s.bin_count;
      }
      __syncthreads();
    }
    const uint32_t b = (uint32_t)(s.bin < 0 ? s.last : s.bin);
    above_mass = s.above_mass;
    above = s.above_count;
    hi -= b << sh;
    const uint32_t reach = (1u << sh) - 1u;
    if (hi - lo > reach) lo = hi - reach;
    if (lo == hi) {
      const Place p = {hi, above, s.bin_count, above_mass, s.bin_mass / s.bin_count};
      __syncthreads();
      return p;
    }
    __syncthreads();
  }
}

// The id of the j-th token (from 1, by id) whose key is `key`; the last one where there are fewer.
template <typename T, bool ALIGNED>
__device__ __noinline__ int find_token(SampleSmem& s, const T* row, int vocab, uint32_t key, uint32_t j) {
  constexpr int PER = Elem<T>::PER16, STEP = 32 * PER;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = (vocab + SP_WARPS * STEP - 1) / (SP_WARPS * STEP) * STEP;
  const long long from = (long long)warp * share, to = from + share < vocab ? from + share : vocab;
  auto matches = [&](long long id) -> uint32_t {
    uint32_t bits = 0;
    if (id < to) {
      float x[PER];
      Elem<T>::unpack(row_vec<T, ALIGNED>(row, (int)id, vocab), x);
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (id + e < to && key_of<T>(x[e]) == key) bits |= 1u << e;
    }
    return bits;
  };
  uint32_t n = 0;
  for (long long i = from; i < to; i += STEP) n += __popc(matches(i + lane * PER));
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  if (lane == 0) s.warp_count[warp] = n;
  if (threadIdx.x == 0) s.bin = 0;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < SP_WARPS; ++w) {
    if (w < warp) before += s.warp_count[w];
    all += s.warp_count[w];
  }
  if (j > all) j = all;
  if (before < j && j <= before + n) {
    uint32_t want = j - before;
    for (long long i = from; i < to; i += STEP) {
      const uint32_t bits = matches(i + lane * PER);
      uint32_t inc = __popc(bits);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += x;
      }
      const uint32_t total = __shfl_sync(0xFFFFFFFFu, inc, 31), excl = inc - __popc(bits);
      if (want <= total) {
        if (excl < want && want <= inc) s.bin = (int)i + lane * PER + __fns(bits, 0, (int)(want - excl));
        break;
      }
      want -= total;
    }
  }
  __syncthreads();
  return s.bin;
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(SP_THREADS) k_sample(SampleArgs a) {
  __shared__ SampleSmem s;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = blockIdx.x, vocab = a.vocab;
  const T* row = static_cast<const T*>(a.logits) + n * a.ld;
  const float t = a.temperature ? __ldg(a.temperature + n) : a.temperature0;
  const float top_p = a.top_p ? __ldg(a.top_p + n) : a.top_p0, min_p = a.min_p ? __ldg(a.min_p + n) : a.min_p0;
  const int top_k = a.top_k ? __ldg(a.top_k + n) : a.top_k0;
  const float u = __ldg(a.u + n);
  for (int i = threadIdx.x; i < (int)(sizeof(ExpTable) / 4); i += SP_THREADS)
    reinterpret_cast<uint32_t*>(&s.tab)[i] = reinterpret_cast<const uint32_t*>(&g_exp_table)[i];
  float m = -INFINITY;
  each<T, ALIGNED>(row, vocab, [&](float z) { m = max_nan(m, z); });
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) s.warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < SP_WARPS; ++w) m = max_nan(m, s.warp_max[w]);
  int token = -1;
  float prob = 0.f;
  // no distribution: a NaN or +inf logit, nothing above -inf, settings or uniforms that are not numbers
  if (fabsf(m) < INFINITY && t >= 0.f && t < INFINITY && top_p == top_p && min_p == min_p && u == u) {
    const uint32_t top = key_of<T>(m);
    if (t == 0.f || top_k == 1 || top_p <= 0.f) {
      token = find_token<T, ALIGNED>(s, row, vocab, top, 1);
      prob = 1.f;
    } else {
      const Weights weight(m, t, 62 - (32 - __clz(vocab - 1)), &s.tab);
      const uint32_t low = key_of<T>(weight.zlow);
      // the kept prefix: the tokens above `key` and the first `equal` of those with it, of mass `mass`
      uint32_t key = low, equal = 0xFFFFFFFFu;
      u64 mass = 0;
      if (top_k > 1 && top_k < vocab) {
        const Place p = descend<T, ALIGNED, true, false>(s, row, vocab, low, top, (u64)top_k, weight);
        key = p.key;
        equal = min((uint32_t)top_k - p.above, p.n_equal);
        mass = p.above_mass + equal * p.w;
      } else {
        u64 sum = 0;
        each<T, ALIGNED>(row, vocab, [&](float z) { sum += weight(z); });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if ((threadIdx.x & 31) == 0) s.warp_mass[threadIdx.x >> 5] = sum;
        __syncthreads();
        for (int w = 0; w < SP_WARPS; ++w) mass += s.warp_mass[w];
        __syncthreads();
      }
      if (top_p < 1.f) {
        u64 want = (u64)ceil((double)top_p * (double)mass);
        if (want < 1) want = 1;
        const Place p = descend<T, ALIGNED, false, false>(s, row, vocab, key, top, want, weight);
        uint32_t j = p.n_equal;
        if (p.w && p.above_mass < want) j = (uint32_t)min((u64)j, (want - p.above_mass + p.w - 1) / p.w);
        if (p.key == key) j = min(j, equal);
        key = p.key;
        equal = j;
        mass = p.above_mass + j * p.w;
      }
      if (min_p > 0.f) {
        // the lowest logit whose weight is min_p of the largest one's
        const double x = (double)m + (double)t * log((double)fminf(min_p, 1.f));
        float f = (float)x;
        if ((double)f < x) f = nextafterf(f, INFINITY);
        const uint32_t least = min(key_at_least<T>(f), top);
        if (least > key) {
          u64 sum = 0;
          each<T, ALIGNED>(row, vocab, [&](float z) {
            if (key_of<T>(z) >= least) sum += weight(z);
          });
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
          if ((threadIdx.x & 31) == 0) s.warp_mass[threadIdx.x >> 5] = sum;
          __syncthreads();
          mass = 0;
          for (int w = 0; w < SP_WARPS; ++w) mass += s.warp_mass[w];
          __syncthreads();
          key = least;
          equal = 0xFFFFFFFFu;
        }
      }
      const double at = fmax((double)u, 0.0) * (double)mass;
      const u64 want = at < (double)mass ? min((u64)at, mass - 1) : mass - 1;
      const Place p = descend<T, ALIGNED, false, true>(s, row, vocab, key, top, want, weight);
      uint32_t j = p.n_equal;
      if (p.w && p.above_mass <= want) j = (uint32_t)min((u64)j, (want - p.above_mass) / p.w + 1);
      if (p.key == key) j = min(j, equal);
      token = find_token<T, ALIGNED>(s, row, vocab, p.key, j);
      prob = (float)((double)p.w / (double)mass);
    }
  }
  if (threadIdx.x == 0) {
    a.token[n] = token;
    if (a.prob) a.prob[n] = prob;
  }
}

}  // namespace

size_t sample_workspace(int, int, int) { return 0; }

cudaError_t launch_sample(const Ctx& c, const SampleArgs& a, int dtype) {
  const int elem = dtype == DH_BF16 ? 2 : 4;
  const bool al = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && (a.N == 1 || a.ld * elem % 16 == 0);
  auto go = [&](auto* kernel) {
    return launch_pdl(c, "sample", kernel, dim3((unsigned)a.N), dim3(SP_THREADS), 0, a);
  };
  if (dtype == DH_BF16) return al ? go(k_sample<__nv_bfloat16, true>) : go(k_sample<__nv_bfloat16, false>);
  return al ? go(k_sample<float, true>) : go(k_sample<float, false>);
}

}  // namespace dh
