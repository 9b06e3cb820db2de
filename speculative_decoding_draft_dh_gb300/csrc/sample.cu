// Sampling one token per row of logits with temperature, top-k, top-p and min-p from a given uniform (definition
// at dh_sample in dh.h).
//
// In the order of a row's tokens by (logit desc, id asc) every filter keeps a prefix, and the drawn token is the
// one at which the prefix's running sum of weights passes u times its mass.  So a token far down the order matters
// only by its share of the row's mass, and that only where no top-k leaves it out.
//   k_sample_scan   the one pass over the logits: the largest of every group of 16 vectors and, of rows whose mass
//                   is needed, every segment's mass.  A warp takes a segment of 128 vectors, so that rows of any
//                   number fill the SMs.  Its bound is HBM (512 rows of 151936 bf16: 25 us, 156 MB at 6.2 TB/s);
//                   with masses, the 25 instructions of a weight (72 us, the issue slots 74% full).
//   k_sample_pick   a block per row.  A bound below which nothing can be drawn: the top_k-th largest group maximum,
//                   or, of rows whose mass is needed, that of the SP_TRY-th, if what is above holds the mass.  The
//                   tokens that reach it are listed, sorted, weighted and summed, and the filters and the draw are
//                   places in that list.  Its bound is the chain of a block's steps, 5 us in one row.
//   k_sample_search the rows whose list would be too long, each by a cluster: a histogram of masses over all
//                   logits, then for each place (of top-k, of top-p, of the draw) the bin that holds it and that
//                   bin's tokens, sorted as a list's.  Where thousands of tokens are equal, or nearly, a bin's tokens
//                   by ranges of their keys instead, until one key is left: its tokens have one weight, so the place
//                   among them is a division, and their order is that of the ids.  Its bound is shared memory's
//                   atomics, two or three of a logit (one flat row 30 us).
// Rows of few segments are scanned by the block that picks, in one launch; rows that the host knows to need no mass
// are searched there too, should they have to be, and a call has two launches.
//
// Which token a uniform falls on hangs on the running sums, so the weights exp((z - max)/T) are integers: fixed
// point with `frac` fraction bits relative to a power of two near the largest, frac = 62 - log2(vocab) (52 at most),
// so that a row's masses fit 64 bits.  Their sums are exact, whatever their order; what is rounded is each weight,
// by half a unit of 2^-frac of the largest (for 2^18 ids half the weight of a token 30 T below the largest logit)
// and by about 2^-28 of itself.  2^(z c), c = log2(e)/T, is taken as 2^(k/64) 2^r with k the rounded 64 z c:
// 2^(k/64) from a table, exact to 2^-29, and 2^r - 1, |r| < 2^-7 + 2^-9, by a cubic in fp32 whose rounding is below
// 2^-29 of the weight; c in two floats, so that z c is exact to 2^-31.
#include "layers.cuh"
#include "rows.cuh"

namespace dh {
namespace {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_BINS = 2048;
constexpr int SP_LIST = 4096;    // tokens listed, at most
constexpr int SP_GROUPS = 2048;  // groups listed, at most
constexpr int SP_FEW = 4 * SP_THREADS;   // tokens of a bin that are sorted, at most
constexpr int SP_SORT = 4 * SP_THREADS;  // of a list
constexpr int SP_RANKED = 128;           // by ranks alone
// A row whose mass is needed is tried with the tokens down to this many groups' maxima before it is searched: the
// usual row at temperature 1 draws from them (one row 15 us; searched 35).  512 rows at top-p 0.95: 155 us with 64,
// 162 with 256, 189 with 64 and then 1024.
constexpr int SP_TRY = 64;
constexpr int SEG_GROUPS = 8;    // groups of a segment: four lanes' vectors each
constexpr int SEG_FRAC = 52;     // fraction bits of a segment's mass, relative to 2^e of its own largest weight

using u64 = unsigned long long;

// ------------------------------------------------------------------ weights

// 2^(j/64): as an integer with 28 fraction bits, and as that value in fp32.
struct ExpTable {
  uint32_t q[64];
  float f[64];
};
// The block's shared memory as one of the structures below, of which each starts with a Scratch.  Every function
// takes it from the symbol itself: through a reference that is passed on the compiler would not know that it is
// shared memory, and atomics and loads on such addresses are several times as slow.
template <class S>
__device__ __forceinline__ S& smem() {
  extern __shared__ __align__(16) unsigned char sample_smem[];
  return *reinterpret_cast<S*>(sample_smem);
}
// What the steps of a block leave for one another.
struct Scratch {
  ExpTable tab;
  u64 warp_mass[SP_WARPS];
  uint32_t warp_count[SP_WARPS];
  float warp_max[SP_WARPS], warp_min[SP_WARPS];
  int bin, last;
  u64 bin_mass, above_mass;
  uint32_t bin_count, above_count;
  uint32_t n_list, n_groups;
  u64 found_mass, found_w;
  u64 found_token;
  uint32_t found_at, found_id;
  uint32_t share[2];  // of a sum over a cluster
  uint32_t n_few;
  u64 few[SP_FEW];  // tokens as in the lists, of a block's share
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

// log2(e) / t in two floats.
struct Rate {
  float hi, lo;
  __device__ __forceinline__ explicit Rate(float t) : hi(1.44269502f / t) {
    lo = (fmaf(-hi, t, 1.44269502f) + 1.92596299e-8f) / t;
  }
};

// The weights of a row whose largest logit is m at temperature t.  z c has to stay below 2^15 for the fp32 form, the
// logits whose weights count above the type's lowest, and 64 c, the steps of a logit, below its largest; beyond that
// (huge logits, tiny and huge temperatures) `far` takes 64-bit arithmetic.
struct Weights {
  Rate c;
  float m, t, zlow;
  int id_bits;      // of the row's ids
  int e_ref, frac;  // the largest weight is in [2^frac, 2^(frac + 1)]
  bool far;
  __device__ __forceinline__ Weights(float m_, float t_, int vocab) : c(t_), m(m_), t(t_) {
    id_bits = 32 - __clz(vocab - 1);
    frac = min(62 - id_bits, SEG_FRAC);
    const float reach = (float)(frac + 2) / c.hi;  // what is lower than m by that much weighs below 2^-(frac + 1)
    far = !(fabsf(m * c.hi) < 32000.f && c.hi < 1e36f && 128.f / c.hi + fabsf(m) < 1e38f);
    zlow = far ? -3.4028234e38f : m - reach;
    e_ref = far ? 0 : (__float_as_int(fmaf(m, c.hi, EXP_MAGIC)) - EXP_MAGIC_BITS) >> 6;
  }
  // far: the weight's 28 bits and how far down they are (64 and more: 0)
  __device__ __noinline__ static uint32_t slow(float z, float m, float t, int* down) {
    const double x = ((double)z - (double)m) * (1.4426950408889634 / (double)t), e = floor(x);
    if (!(e > -64.0)) {
      *down = 64;
      return 0;
    }
    *down = -(int)e;
    return (uint32_t)rint(exp2(x - e) * 268435456.0);
  }
  // not far: the weight in 64ths of an octave, rounded
  __device__ __forceinline__ int step(float z) const {
    return __float_as_int(fmaf(z, c.hi, EXP_MAGIC)) - EXP_MAGIC_BITS;
  }
  // 28 fraction bits to frac, and down, rounded; z is at least zlow, so that the shift is at most 62
  __device__ __forceinline__ u64 scaled(uint32_t q, int down) const {
    return ((((u64)q << 32) >> min(59 - frac + down, 63)) + 1) >> 1;
  }
  // not far, z at least zlow
  __device__ __forceinline__ u64 near(float z) const {
    const float k = fmaf(z, c.hi, EXP_MAGIC), kf = k - EXP_MAGIC;
    const float r = fmaf(z, c.lo, fmaf(z, c.hi, -kf));
    const int ki = step(z), j = ki & 63;
    // 2^r - 1 by its series
    const float x = r * fmaf(r, fmaf(r, 0.0555041087f, 0.240226507f), 0.693147181f);
    // added to 1.5 2^23, which rounds to an integer in the low bits; |tab.f x| < 2^22
    const ExpTable& tab = smem<Scratch>().tab;
    const uint32_t q = tab.q[j] + (uint32_t)(__float_as_int(fmaf(tab.f[j], x, 12582912.f)) - 0x4B400000);
    return scaled(q, e_ref - (ki >> 6));
  }
  __device__ __forceinline__ u64 operator()(float z) const {
    if (!(z >= zlow)) return 0;
    if (__builtin_expect(!far, 1)) return near(z);
    int down;
    const uint32_t q = slow(z, m, t, &down);
    return scaled(q, down);
  }
};

// x mass rounded down, and whether something was left over, exactly, for 0 <= x < 1.
__device__ __forceinline__ u64 times(float x, u64 mass, bool* rest) {
  const uint32_t bits = __float_as_uint(x);
  const u64 n = (bits & 0x7FFFFFu) | 0x800000u;
  const int s = 150 - (int)(bits >> 23);  // x = n 2^-s
  const u64 lo = n * mass, hi = __umul64hi(n, mass);
  *rest = x > 0.f;
  if (bits < 0x00800000u || s > 87) return 0;  // below 2^-87
  if (s >= 64) {
    *rest = lo != 0 || (s > 64 && (hi << (128 - s)) != 0);
    return hi >> (s - 64);
  }
  *rest = (lo << (64 - s)) != 0;
  return (hi << (64 - s)) | (lo >> s);
}

// Order-preserving keys: of fp32 logits 32 bits, of bf16 logits 16.
template <typename T>
__device__ __forceinline__ uint32_t key_of(float z) {
  return sizeof(T) == 4 ? fkey(z) : fkey(z) >> 16;
}
template <typename T>
__device__ __forceinline__ float value_of(uint32_t key) {
  if (sizeof(T) == 4) return fkey_inv(key);
  return fkey_inv((key & 0x8000u) ? key << 16 : (key << 16) | 0xFFFFu);
}
// ------------------------------------------------------------------ the pass over the logits

// A segment's mass, in units of 2^(e - SEG_FRAC).
struct SegMass {
  u64 mass;
  int e;
  int pad;
};

// What of a row's settings asks for: its whole mass (no top-k bounds what is kept, and what is kept or drawn is a
// share of all).
__device__ __forceinline__ bool needs_mass(float t, int top_k, float top_p, float min_p, int vocab) {
  return t > 0.f && !(top_k >= 1 && top_k < vocab) && top_p > 0.f && (top_p < 1.f || !(min_p > 0.f));
}

// The table of 2^(j/64), a copy for each of 16 lanes so that a warp's look-ups do not meet in a bank.
struct ScanTable {
  uint2 e[64 * 16];
};
__device__ __forceinline__ void fill_table(ScanTable& t, int threads) {
  for (int i = threadIdx.x; i < 64 * 16; i += threads)
    t.e[i] = make_uint2(g_exp_table.q[i >> 4], __float_as_uint(g_exp_table.f[i >> 4]));
}

// Segment sgi of a row by one warp: the maxima of its groups (lanes 4 g .. 4 g + 3 have group g's) and, if `mass`,
// its mass at temperature t.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void scan_segment(const T* row, int sgi, int vocab, float t, bool mass, const ScanTable& tab,
                                             float* gmax, SegMass* seg) {
  constexpr int PER = Elem<T>::PER16;
  const int lane = threadIdx.x & 31;
  const int id0 = sgi * row_seg<T>() + lane * PER;
  uint4 u[ROW_SEG_VECS];
#pragma unroll
  for (int v = 0; v < ROW_SEG_VECS; ++v) u[v] = row_vec<T, ALIGNED>(row, id0 + v * 32 * PER, vocab);
  float m = vec_max<T>(u);
  m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  if ((lane & 3) == 0) gmax[sgi * SEG_GROUPS + (lane >> 2)] = m;
  if (!mass) return;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const Rate c(t);
  // (what is lower than m by `reach` counts as 0)
  const float ch = c.hi, cl = c.lo, reach = (float)(SEG_FRAC + 2) / ch;
  u64 sum = 0;
  int e_ref = -0x40000000;
  // beyond, and so beyond the limits of Weights: the row's weights are taken in 64 bits by the block that picks, or
  // its largest logit is so far above this segment's that their weights are 0
  if (fabsf(m * ch) < 32700.f && ch < 1e38f && 128.f / ch + fabsf(m) < 3.3e38f) {
    e_ref = (__float_as_int(fmaf(m, ch, EXP_MAGIC)) - EXP_MAGIC_BITS) >> 6;
    const float low = m - reach;
    const uint2* tb = tab.e + (lane & 15);
    const f32x2 cc = pack2(ch, ch), cd = pack2(cl, cl), magic = pack2(EXP_MAGIC, EXP_MAGIC);
    const f32x2 none = pack2(-1.f, -1.f);
    const f32x2 c3 = pack2(0.0555041087f, 0.0555041087f), c2 = pack2(0.240226507f, 0.240226507f),
                c1 = pack2(0.693147181f, 0.693147181f);
    const int base = e_ref + (EXP_MAGIC_BITS >> 6) + 8;  // with 2^24 of the 2^52, counted from bit 32
#pragma unroll
    for (int v = 0; v < ROW_SEG_VECS; ++v) {
      float x[PER];
      Elem<T>::unpack(u[v], x);
#pragma unroll
      for (int q = 0; q < PER; q += 2) {
        const f32x2 z = pack2(fmaxf(x[q], low), fmaxf(x[q + 1], low));
        const f32x2 k = fma2(z, cc, magic);
        const f32x2 r = fma2(z, cd, fma2(z, cc, fma2(k, none, magic)));  // (magic - k is exact)
        const f32x2 y = mul2(r, fma2(r, fma2(r, c3, c2), c1));
        float ka, kb, ya, yb;
        unpack2(k, ka, kb);
        unpack2(y, ya, yb);
        auto one = [&](float kx, float yx) {
          const int ki = __float_as_int(kx);
          const uint2 w = tb[(ki & 63) * 16];
          const uint32_t n = w.x + (uint32_t)(__float_as_int(fmaf(__uint_as_float(w.y), yx, 12582912.f)) - 0x4B400000);
          // n 2^24 >> (e_ref - e), from n 2^32
          sum += ((u64)n << 32) >> (base - (ki >> 6));  // at most 63: z is at least low
        };
        one(ka, ya);
        one(kb, yb);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) seg[sgi] = {sum, e_ref, 0};
}

constexpr int SC_THREADS = 256;
constexpr int SC_BLOCKS = 5;  // of an SM

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(SC_THREADS, SC_BLOCKS) k_sample_scan(SampleArgs a, int n_seg, float* gmax,
                                                                       SegMass* segs) {
  __shared__ ScanTable tab;
  fill_table(tab, SC_THREADS);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the picking kernel follows
  const unsigned nw = gridDim.x * (SC_THREADS / 32);
  const unsigned long long items = (unsigned long long)a.N * n_seg;
  for (unsigned long long g = blockIdx.x * (SC_THREADS / 32) + (threadIdx.x >> 5); g < items; g += nw) {
    int n, sgi;
    if (items < 0x7F000000ull) {
      n = (int)((unsigned)g / (unsigned)n_seg);
      sgi = (int)((unsigned)g - (unsigned)n * (unsigned)n_seg);
    } else {
      n = (int)(g / n_seg);
      sgi = (int)(g - (unsigned long long)n * n_seg);
    }
    const float t = a.temperature ? __ldg(a.temperature + n) : a.temperature0;
    const bool mass = needs_mass(t, a.top_k ? __ldg(a.top_k + n) : a.top_k0, a.top_p ? __ldg(a.top_p + n) : a.top_p0,
                                 a.min_p ? __ldg(a.min_p + n) : a.min_p0, a.vocab);
    scan_segment<T, ALIGNED>(static_cast<const T*>(a.logits) + n * a.ld, sgi, a.vocab, t, mass, tab,
                             gmax + (long long)n * n_seg * SEG_GROUPS, segs + (long long)n * n_seg);
  }
}

// ------------------------------------------------------------------ the search

// A histogram over a range of keys: masses in two words, counts.
struct __align__(16) Bins {
  uint32_t lo[SP_BINS], hi[SP_BINS], count[SP_BINS];
  __device__ __forceinline__ u64 mass(int b) const { return ((u64)hi[b] << 32) | lo[b]; }
  // n tokens (0: not counted) of mass w
  __device__ __forceinline__ void add(uint32_t b, u64 w, uint32_t n) {
    if (n) atomicAdd(&count[b], n);
    const uint32_t x = (uint32_t)w;
    uint32_t h = (uint32_t)(w >> 32);
    // (there is no 64-bit addition in shared memory)
    if (x) h += atomicAdd(&lo[b], x) > ~x;
    if (h) atomicAdd(&hi[b], h);
  }
};

struct SampleSmem : Scratch {
  static constexpr int RANKS = 1;  // blocks of a search
  __device__ __forceinline__ u64* row_few() { return few; }
  __device__ __forceinline__ Bins& local(int level) { return bins[level]; }
  union {
    Bins bins[2];  // of the whole range, of a part of it
    struct {
      uint32_t group_count[SP_BINS], groups[SP_GROUPS];
    };
  };
  u64 list[SP_LIST];  // key << 32 | ~id: the order is that of these numbers, descending
};
// Blocks of a cluster: 512 flat rows 534 us, one 61, 512 rows at top-p 0.95 154.  More rows at once would be faster with 2
// (405, 86 and 166), one with 8 (1057, 56 and 225); a batch of which some rows are searched is the usual case.
constexpr int SS_RANKS = 4;
struct SearchSmem : Scratch {
  static constexpr int RANKS = SS_RANKS;
  u64 all_few[SP_FEW];  // of the row
  __device__ __forceinline__ u64* row_few() { return all_few; }
  __device__ __forceinline__ Bins& local(int) { return own; }
  Bins own;      // of this block's share of the row
  Bins bins[2];  // of the whole row
};

// A place in the order: all tokens above `key`, of which there are `above` with mass `above_mass`, and the tokens
// of that key: n_equal, each of weight w.
struct Place {
  uint32_t key, above, n_equal;
  u64 above_mass, w;
};

// A block's share of a row: the ids [from, to), whole steps of a warp but for the row's end; or the listed tokens.
struct Share {
  int from, to;
  bool listed;
};
template <typename T, int RANKS>
__device__ __forceinline__ Share share_of_row(int vocab) {
  if (RANKS == 1) return {0, vocab, false};
  constexpr int STEP = 32 * Elem<T>::PER16;
  const int each = (vocab + RANKS * STEP - 1) / (RANKS * STEP) * STEP, from = min((int)cluster_rank() * each, vocab);
  return {from, min(from + each, vocab), false};
}

// f(value, id) of every token of the list.
template <typename T, typename F>
__device__ __forceinline__ void each_listed(F f) {
  const SampleSmem& s = smem<SampleSmem>();
  for (int i = threadIdx.x; i < (int)s.n_list; i += SP_THREADS) {
    const u64 x = s.list[i];
    f(value_of<T>((uint32_t)(x >> 32)), ~(uint32_t)x);
  }
}

// f(value) of every logit of the share that is in [from, to] (finite numbers).
template <typename T, bool ALIGNED, typename F>
__device__ __forceinline__ void each(const T* row, Share part, float from, float to, F f) {
  constexpr int PER = Elem<T>::PER16, AHEAD = 4;
  for (int id0 = part.from + threadIdx.x * PER; id0 < part.to; id0 += AHEAD * SP_THREADS * PER) {
    uint4 u[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int id = id0 + q * SP_THREADS * PER;
      u[q] = make_uint4(NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD);
      if (id < part.to) u[q] = row_vec<T, ALIGNED>(row, id, part.to);
    }
#pragma unroll 1
    for (int q = 0; q < AHEAD; ++q) {
      float x[PER];
      Elem<T>::unpack(q == 0 ? u[0] : q == 1 ? u[1] : q == 2 ? u[2] : u[3], x);
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (x[e] >= from && x[e] <= to) f(x[e]);
    }
  }
}

// Which elements of a vector are in [from, to], by two comparisons per word.
template <typename T>
struct Within {
  float from, to;
  __device__ __forceinline__ Within(float f, float t) : from(f), to(t) {}
  __device__ __forceinline__ uint32_t operator()(const uint4& u) const {
    float x[4];
    Elem<T>::unpack(u, x);
    uint32_t hits = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) hits |= (x[e] >= from && x[e] <= to ? 1u : 0u) << e;
    return hits;
  }
};
template <>
struct Within<__nv_bfloat16> {
  __nv_bfloat162 from, to;  // bf16 values
  __device__ __forceinline__ Within(float f, float t) : from(__float2bfloat162_rn(f)), to(__float2bfloat162_rn(t)) {}
  __device__ __forceinline__ uint32_t operator()(const uint4& u) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[q]);
      m[q] = __hge2_mask(x, from) & __hle2_mask(x, to);
    }
    if (!((m[0] | m[1]) | (m[2] | m[3]))) return 0;
    uint32_t hits = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) hits |= ((m[q] & 1u) | ((m[q] >> 15) & 2u)) << (2 * q);
    return hits;
  }
};
// Element e of a vector.
template <typename T>
__device__ __forceinline__ float element(const uint4& u, int e) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(e < 2 ? (e == 0 ? u.x : u.y) : (e == 2 ? u.z : u.w));
  } else {
    const uint32_t w = e < 4 ? (e < 2 ? u.x : u.y) : (e < 6 ? u.z : u.w);
    return __uint_as_float((e & 1) ? w & 0xFFFF0000u : w << 16);
  }
}
// f(value, id) as `each`, where few are: from and to are values of T.
template <typename T, bool ALIGNED, typename F>
__device__ __forceinline__ void each_of_few(const T* row, Share part, float from, float to, F f) {
  constexpr int PER = Elem<T>::PER16, AHEAD = 4;
  const Within<T> within(from, to);
  for (int id0 = part.from + threadIdx.x * PER; id0 < part.to; id0 += AHEAD * SP_THREADS * PER) {
    uint4 u[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int id = id0 + q * SP_THREADS * PER;
      u[q] = make_uint4(NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD);
      if (id < part.to) u[q] = row_vec<T, ALIGNED>(row, id, part.to);
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
      for (uint32_t hits = within(u[q]); hits; hits &= hits - 1) {
        const int e = __ffs(hits) - 1;
        f(element<T>(u[q], e), (uint32_t)(id0 + q * SP_THREADS * PER + e));
      }
  }
}

// What a place is searched by: a number of tokens, a mass, or more than a mass.  (Arguments, not template parameters:
// a row's searches then share their code, which comes from memory the first time.)
enum Goal { TOKENS, MASS, ABOVE };
__device__ __forceinline__ bool reached(Goal goal, u64 want, u64 mass, uint32_t count) {
  return goal == TOKENS ? count >= want : goal == ABOVE ? mass > want : mass >= want;
}

// The bin, from the top down, in which `want` is reached, counted on from `above` tokens of `above_mass`; the last bin
// that is not empty where it is not, -1 where all are empty.
struct Histogram {
  int bin;
  uint32_t above, count;
  u64 above_mass, mass;
};
__device__ __forceinline__ int bin_shift(uint32_t lo, uint32_t hi) {
  const int bits = 32 - __clz(hi - lo);
  return bits > 11 ? bits - 11 : 0;
}

// Tokens of one bin, added together: of rows of equal or nearly equal logits neighbours meet in a bin, and a warp's
// atomics on one address take turns (512 rows of equal logits 1.7 ms, 2.5 without).
struct Pending {
  int bin = -1;
  u64 mass = 0;
  uint32_t count = 0;
  __device__ __forceinline__ void add(Bins& bins, int b, u64 w, uint32_t n, bool counted) {
    if (b != bin) {
      flush(bins, counted);
      bin = b;
      mass = 0;
      count = 0;
    }
    mass += w;
    count += n;
  }
  __device__ __forceinline__ void flush(Bins& bins, bool counted) const {
    if (bin >= 0) bins.add(bin, mass, counted ? count : 0);
  }
};

// The bins of a row's first histogram: 32nds of an octave of the weights (linear in the logits, so that neighbouring
// tokens seldom meet in a bin), or, where weights are far, ranges of keys.
struct Coarse {
  int top;        // step of the largest weight
  uint32_t lo, hi;
  int sh;         // far: of the keys
  bool far;
  template <typename T>
  __device__ __forceinline__ int bin(float z, const Weights& weight) const {
    return far ? (int)((hi - key_of<T>(z)) >> sh) : (top - weight.step(z)) >> 1;
  }
  // The range of keys that holds a bin's tokens (and others).
  template <typename T>
  __device__ __forceinline__ void keys(int b, const Weights& weight, uint32_t* from, uint32_t* to) const {
    if (far) {
      const uint32_t reach = (1u << sh) - 1u;
      *to = hi - ((uint32_t)b << sh);
      *from = *to - lo > reach ? *to - reach : lo;
    } else {
      // half a step more on either side covers the roundings
      const float steps = 64.f * weight.c.hi;
      const float z1 = (float)(top - 2 * b + 1) / steps, z0 = (float)(top - 2 * b - 2) / steps;
      *from = max(lo, min(key_of<T>(z0), hi));
      *to = min(hi, max(key_of<T>(z1), *from));
    }
  }
};

// bins[level] = the sum of the cluster's local bins.
template <class S>
__device__ __forceinline__ void merge_bins(int level) {
  if constexpr (S::RANKS == 1) {
    __syncthreads();  // they are the same
  } else {
    S& s = smem<S>();
    const Bins& local = s.local(level);
    Bins& out = s.bins[level];
    static_assert(SP_BINS == 4 * SP_THREADS, "a thread has four bins");
    cluster_sync();
    const int b = threadIdx.x;
    u64 m[4] = {0, 0, 0, 0};
    uint4 c = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (uint32_t r = 0; r < S::RANKS; ++r) {
      const uint4 l = ld_cluster(reinterpret_cast<const uint4*>(local.lo) + b, r);
      const uint4 h = ld_cluster(reinterpret_cast<const uint4*>(local.hi) + b, r);
      const uint4 n = ld_cluster(reinterpret_cast<const uint4*>(local.count) + b, r);
      m[0] += ((u64)h.x << 32) | l.x;
      m[1] += ((u64)h.y << 32) | l.y;
      m[2] += ((u64)h.z << 32) | l.z;
      m[3] += ((u64)h.w << 32) | l.w;
      c.x += n.x;
      c.y += n.y;
      c.z += n.z;
      c.w += n.w;
    }
    reinterpret_cast<uint4*>(out.lo)[b] = make_uint4((uint32_t)m[0], (uint32_t)m[1], (uint32_t)m[2], (uint32_t)m[3]);
    reinterpret_cast<uint4*>(out.hi)[b] =
        make_uint4((uint32_t)(m[0] >> 32), (uint32_t)(m[1] >> 32), (uint32_t)(m[2] >> 32), (uint32_t)(m[3] >> 32));
    reinterpret_cast<uint4*>(out.count)[b] = c;
    cluster_sync();  // `local` has been read
  }
}
template <class S>
__device__ __forceinline__ void clear_bins(int level) {
  Bins& bins = smem<S>().local(level);
  for (int b = threadIdx.x; b < SP_BINS / 4; b += SP_THREADS)
    reinterpret_cast<uint4*>(bins.lo)[b] = reinterpret_cast<uint4*>(bins.hi)[b] =
        reinterpret_cast<uint4*>(bins.count)[b] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
}
// Those of a share with a weight, where weights are near.  A vector's tokens side by side: an atomic's result comes
// after many instructions, and one after the other a row of 151936 flat logits takes 25 us by four blocks.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void add_near(const T* row, Share part, Coarse coarse, const Weights& weight, Bins& bins,
                                         bool counted) {
  constexpr int PER = Elem<T>::PER16, AHEAD = 4;
  Pending same;
  for (int id0 = part.from + threadIdx.x * PER; id0 < part.to; id0 += AHEAD * SP_THREADS * PER) {
    uint4 u[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int id = id0 + q * SP_THREADS * PER;
      u[q] = make_uint4(NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD);
      if (id < part.to) u[q] = row_vec<T, ALIGNED>(row, id, part.to);
    }
#pragma unroll 1
    for (int q = 0; q < AHEAD; ++q) {
      float x[PER];
      Elem<T>::unpack(q == 0 ? u[0] : q == 1 ? u[1] : q == 2 ? u[2] : u[3], x);
      int b[PER];
      uint32_t lo[PER], hi[PER];
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const float z = fmaxf(x[e], weight.zlow);
        const u64 w = weight.near(z);
        b[e] = x[e] >= weight.zlow ? (coarse.top - weight.step(z)) >> 1 : -1;
        lo[e] = (uint32_t)w;
        hi[e] = (uint32_t)(w >> 32);
      }
      bool one = true;
#pragma unroll
      for (int e = 1; e < PER; ++e) one &= b[e] == b[0];
      if (one) {
        if (b[0] < 0) continue;
        u64 w = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) w += ((u64)hi[e] << 32) | lo[e];
        same.add(bins, b[0], w, PER, counted);
        continue;
      }
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (b[e] >= 0) hi[e] += atomicAdd(&bins.lo[b[e]], lo[e]) > ~lo[e];
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (b[e] >= 0 && hi[e]) atomicAdd(&bins.hi[b[e]], hi[e]);
      if (counted) {
#pragma unroll
        for (int e = 0; e < PER; ++e)
          if (b[e] >= 0) atomicAdd(&bins.count[b[e]], 1u);
      }
    }
  }
  same.flush(bins, counted);
}
// All tokens with a weight, by the coarse bins, into bins[0].
template <typename T, bool ALIGNED, class S>
__device__ __noinline__ void fill_coarse(const T* row, Share part, Coarse coarse, Weights weight, bool counted) {
  clear_bins<S>(0);
  Bins& local = smem<S>().local(0);
  auto add = [&](float z, uint32_t = 0) { local.add(coarse.bin<T>(z, weight), weight(z), counted ? 1u : 0u); };
  if (S::RANKS == 1 && part.listed) each_listed<T>(add);
  else if (!weight.far) add_near<T, ALIGNED>(row, part, coarse, weight, local, counted);
  else each<T, ALIGNED>(row, part, weight.zlow, weight.m, add);
  merge_bins<S>(0);
}
// Those of one coarse bin with keys [lo, hi], by ranges of keys, into bins[1].
template <typename T, bool ALIGNED, class S>
__device__ __noinline__ void fill_fine(const T* row, Share part, Coarse coarse, int bin, uint32_t lo, uint32_t hi,
                                       Weights weight) {
  clear_bins<S>(1);
  Bins& local = smem<S>().local(1);
  const int sh = bin_shift(lo, hi);
  Pending same;
  each_of_few<T, ALIGNED>(row, part, value_of<T>(lo), value_of<T>(hi), [&](float z, uint32_t) {
    if (coarse.bin<T>(z, weight) == bin) same.add(local, (int)((hi - key_of<T>(z)) >> sh), weight(z), 1u, true);
  });
  same.flush(local, true);
  merge_bins<S>(1);
}
template <class S>
__device__ __noinline__ Histogram find_bin(int level, uint32_t above, u64 above_mass, u64 want, Goal goal) {
  S& s = smem<S>();
  const Bins& bins = s.bins[level];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    s.bin = s.last = -1;
    s.bin_mass = s.bin_count = 0;
    s.above_mass = above_mass;
    s.above_count = above;
  }
  // inclusive sums over the bins, four to a thread
  constexpr int OWN = SP_BINS / SP_THREADS;
  u64 m = 0;
  uint32_t c = 0;
  const int b0 = threadIdx.x * OWN;
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    m += bins.mass(b0 + q);
    c += bins.count[b0 + q];
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
  auto found = [&](int b, u64 mass_before, uint32_t count_before) {
    s.bin_mass = bins.mass(b);
    s.bin_count = bins.count[b];
    s.above_mass = mass_before;
    s.above_count = count_before;
  };
  int last = -1;
  u64 last_mass = 0;
  uint32_t last_count = 0;
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    const u64 mb = bins.mass(b0 + q);
    const uint32_t cb = bins.count[b0 + q];
    if (cb || mb) {
      last = b0 + q;
      last_mass = ma;
      last_count = ca;
    }
    if (!reached(goal, want, ma, ca) && reached(goal, want, ma + mb, ca + cb)) {
      s.bin = b0 + q;
      found(b0 + q, ma, ca);
    }
    ma += mb;
    ca += cb;
  }
  if (last >= 0) atomicMax(&s.last, last);
  __syncthreads();
  // where the sums never reach it: the last bin that is not empty
  if (s.bin < 0 && last >= 0 && last == s.last) found(last, last_mass, last_count);
  __syncthreads();
  const Histogram h = {s.bin < 0 ? s.last : s.bin, s.above_count, s.bin_count, s.above_mass, s.bin_mass};
  __syncthreads();
  return h;
}

// The first place at which `want` is reached, the last place where it is not.  bins[0] is the row's coarse histogram.
template <typename T, bool ALIGNED, class S>
__device__ __noinline__ Place descend(const T* row, Share part, Coarse coarse, u64 want, Goal goal, Weights weight) {
  Place p = {};
  Histogram h = find_bin<S>(0, 0, 0, want, goal);
  const int bin = h.bin;
  uint32_t lo, hi;
  coarse.keys<T>(bin, weight, &lo, &hi);
  for (;;) {
    p.above_mass = h.above_mass;
    p.above = h.above;
    fill_fine<T, ALIGNED, S>(row, part, coarse, bin, lo, hi, weight);
    const int sh = bin_shift(lo, hi);
    h = find_bin<S>(1, p.above, p.above_mass, want, goal);
    if (h.bin < 0) {  // none of the bin's tokens: no place
      p.key = hi;
      return p;
    }
    hi -= (uint32_t)h.bin << sh;
    const uint32_t reach = (1u << sh) - 1u;
    if (hi - lo > reach) lo = hi - reach;
    if (lo == hi) {
      p.above_mass = h.above_mass;
      p.above = h.above;
      p.key = hi;
      p.n_equal = h.count;
      p.w = h.count ? h.mass / h.count : 0;
      return p;
    }
  }
}

// The id of the j-th token (from 1, by id) whose key is `key`, the last one where there are fewer, -1 where there is
// none; ELSEWHERE in the blocks of a cluster that have nothing to say.
constexpr int ELSEWHERE = -2;
template <typename T, bool ALIGNED, int RANKS>
__device__ __noinline__ int find_token(const T* row, Share part, uint32_t key, uint32_t j) {
  Scratch& s = smem<Scratch>();
  constexpr int PER = Elem<T>::PER16, STEP = 32 * PER;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (part.to - part.from + SP_WARPS * STEP - 1) / (SP_WARPS * STEP) * STEP;
  const int from = min(part.from + warp * each, part.to), to = min(from + each, part.to);
  const Within<T> within(value_of<T>(key), value_of<T>(key));  // (a finite number, so not what lies past the row's end)
  auto matches = [&](int id) -> uint32_t { return id < to ? within(row_vec<T, ALIGNED>(row, id, to)) : 0u; };
  uint32_t n = 0;
#pragma unroll 4
  for (int i = from; i < to; i += STEP) n += __popc(matches(i + lane * PER));
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  if (lane == 0) s.warp_count[warp] = n;
  if (threadIdx.x == 0) s.bin = RANKS > 1 ? ELSEWHERE : -1;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < SP_WARPS; ++w) {
    if (w < warp) before += s.warp_count[w];
    all += s.warp_count[w];
  }
  if constexpr (RANKS > 1) {
    if (threadIdx.x == 0) s.share[0] = all;
    cluster_sync();
    uint32_t total = 0;
    for (uint32_t r = 0; r < RANKS; ++r) {
      const uint32_t x = ld_cluster(&s.share[0], r);
      if (r < cluster_rank()) before += x;
      total += x;
    }
    all = total;
    cluster_sync();
  }
  if (all == 0) return RANKS > 1 && cluster_rank() != 0 ? ELSEWHERE : -1;
  j = min(max(j, 1u), all);
  if (before < j && j <= before + n) {
    uint32_t want = j - before;
    for (int i = from; i < to; i += STEP) {
      const uint32_t bits = matches(i + lane * PER);
      uint32_t inc = __popc(bits);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += x;
      }
      const uint32_t total = __shfl_sync(0xFFFFFFFFu, inc, 31), excl = inc - __popc(bits);
      if (want <= total) {
        if (excl < want && want <= inc) s.bin = i + lane * PER + __fns(bits, 0, (int)(want - excl));
        break;
      }
      want -= total;
    }
  }
  __syncthreads();
  return s.bin;
}

// w / mass, 0 < w <= mass, within 2^-24 and a little: the quotient of the rounded numbers, corrected by what the
// roundings and the division left over.  (Double precision would take a warp a microsecond.)
__device__ __forceinline__ float share(u64 w, u64 mass) {
  const float a = __ull2float_rn(w), b = __ull2float_rn(mass), q = a / b;
  const float da = __ll2float_rn((long long)(w - (u64)a)), db = __ll2float_rn((long long)(mass - (u64)b));
  return q + (fmaf(-q, b, a) + fmaf(-q, db, da)) / b;
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ u64 block_mass(u64 x) {
  Scratch& s = smem<Scratch>();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  if ((threadIdx.x & 31) == 0) s.warp_mass[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
  for (int w = 0; w < SP_WARPS; ++w) x += s.warp_mass[w];
  __syncthreads();
  return x;
}
// Sum over the threads before this one.
__device__ __forceinline__ u64 mass_before(u64 x) {
  Scratch& s = smem<Scratch>();
  u64 inc = x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s.warp_mass[warp] = inc;
  __syncthreads();
  u64 before = inc - x;
  for (int w = 0; w < warp; ++w) before += s.warp_mass[w];
  return before;
}

// The settings of a row and what is known of it.
struct RowState {
  uint32_t top;    // key of the largest logit
  uint32_t low;    // of the smallest logit with a weight
  uint32_t least;  // of a logit that is below every one that min-p keeps (0: it leaves out none)
  u64 w_min;       // the smallest weight that min-p keeps
  int top_k;       // 0: none
  float top_p, u;
  u64 mass;        // of the row, where no top-k bounds it (0: not known)
};

// The place of a draw in a mass: the token whose running sum is the first above it.
__device__ __forceinline__ u64 draw_at(float u, u64 mass) {
  if (!(u > 0.f)) return 0;
  bool rest;
  return u < 1.f ? times(u, mass, &rest) : mass - 1;
}
// The mass that top-p asks for.
__device__ __forceinline__ u64 share_of(float p, u64 mass) {
  bool rest;
  const u64 want = times(p, mass, &rest) + rest;
  return want < 1 ? 1 : want;
}

// Sum over the block, or the cluster, that searches a row; every thread gets it.
template <class S>
__device__ __forceinline__ u64 row_mass(u64 x) {
  u64 mass = block_mass(x);
  if constexpr (S::RANKS > 1) {
    S& s = smem<S>();
    if (threadIdx.x == 0) {
      s.share[0] = (uint32_t)mass;
      s.share[1] = (uint32_t)(mass >> 32);
    }
    cluster_sync();
    mass = 0;
    for (uint32_t k = 0; k < S::RANKS; ++k)
      mass += ((u64)ld_cluster(&s.share[1], k) << 32) | ld_cluster(&s.share[0], k);
    cluster_sync();
  }
  return mass;
}
// The mass of the tokens that min-p keeps.
template <typename T, bool ALIGNED, class S>
__device__ __noinline__ u64 mass_of_heavy(const T* row, Share part, u64 w_min, uint32_t least, Weights weight) {
  u64 sum = 0;
  auto add = [&](float z, uint32_t = 0) {
    const u64 w = weight(z);
    if (w >= w_min) sum += w;
  };
  if (S::RANKS == 1 && part.listed) each_listed<T>(add);
  else each<T, ALIGNED>(row, part, fmaxf(value_of<T>(least), weight.zlow), weight.m, add);
  return row_mass<S>(sum);
}

// The first n <= OWN SP_THREADS of `a` (shared memory) in descending order; they are distinct.  A few are ranked among
// one another; more are counted by ranges of their keys or values first, of one key by ranges of ids, so that most
// ranges have a token or none, and then ranked among their range's.  (One list of 20: a call of 9.9 us by ranks, 10.4
// by ranges; 77 lists of 565: 26 us by ranges, 39 by a bitonic network.)
template <typename T, int OWN>
__device__ __forceinline__ void sort_few(u64* a, int n, int id_bits, Bins& bins) {
  Scratch& s = smem<Scratch>();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (n <= SP_RANKED) {
    const u64 x = (int)threadIdx.x < n ? a[threadIdx.x] : 0;
    int rank = 0;
    if ((int)threadIdx.x < n) {
#pragma unroll 4
      for (int k = 0; k < n; ++k) rank += a[k] > x;
    }
    __syncthreads();
    if ((int)threadIdx.x < n) a[rank] = x;
    __syncthreads();
    return;
  }
  u64 x[OWN];
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    const int i = threadIdx.x + q * SP_THREADS;
    x[q] = i < n ? a[i] : 0;
    if (i < n) {
      lo = min(lo, (uint32_t)(x[q] >> 32));
      hi = max(hi, (uint32_t)(x[q] >> 32));
    }
  }
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  if (lane == 0) s.warp_mass[warp] = ((u64)hi << 32) | lo;
  reinterpret_cast<uint4*>(bins.count)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  static_assert(SP_WARPS <= 32 && SP_BINS == 4 * SP_THREADS, "a lane per warp, four bins per thread");
  const u64 range = lane < SP_WARPS ? s.warp_mass[lane] : 0xFFFFFFFFull;
  lo = __reduce_min_sync(0xFFFFFFFFu, (uint32_t)range);
  hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(range >> 32));
  // by keys and ids where a bin has one key, else by values: a wide range's keys are mostly those of numbers near 0
  const int sh = bin_shift(lo, hi), more = max(11 - (32 - __clz(hi - lo)), 0), id_sh = max(id_bits - more, 0);
  const float largest = value_of<T>(hi), reach = largest - value_of<T>(lo);
  const float per_bin = reach < INFINITY ? (SP_BINS - 1) / reach : 0.f;
  uint32_t at[OWN], slot[OWN];
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    const uint32_t key = (uint32_t)(x[q] >> 32);
    if (sh == 0) at[q] = ((hi - key) << more) + (~(uint32_t)x[q] >> id_sh);
    else at[q] = min((uint32_t)((largest - value_of<T>(key)) * per_bin), SP_BINS - 1u);
    if ((int)threadIdx.x + q * SP_THREADS < n) slot[q] = atomicAdd(&bins.count[at[q]], 1u);
  }
  __syncthreads();
  const uint4 c = reinterpret_cast<const uint4*>(bins.count)[threadIdx.x];
  const uint32_t own = c.x + c.y + c.z + c.w;
  uint32_t before = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, before, o);
    if (lane >= o) before += y;
  }
  if (lane == 31) s.warp_count[warp] = before;
  before -= own;
  __syncthreads();
  before += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s.warp_count[lane] : 0u);
  reinterpret_cast<uint4*>(bins.lo)[threadIdx.x] =
      make_uint4(before, before + c.x, before + c.x + c.y, before + c.x + c.y + c.z);
  __syncthreads();
  uint32_t count[OWN];
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    count[q] = 0;
    if ((int)threadIdx.x + q * SP_THREADS < n) {
      count[q] = bins.count[at[q]];
      at[q] = bins.lo[at[q]];
      a[at[q] + slot[q]] = x[q];
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    slot[q] = 0;
    if (count[q] > 1)
      for (uint32_t k = 0; k < count[q]; ++k) slot[q] += a[at[q] + k] > x[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < OWN; ++q)
    if (count[q] > 1) a[at[q] + slot[q]] = x[q];
  __syncthreads();
}

// The token (as in the lists) at which `want` is reached, of the tokens of coarse bin h.bin, the running sum up to and
// with it, and its weight; the bin's last one where it is not.  False where the bin has more tokens than are sorted, or
// none.
struct Cut {
  u64 token, mass, w;
};
template <typename T, bool ALIGNED, class S>
__device__ __noinline__ bool resolve(const T* row, Share part, Coarse coarse, Histogram h, u64 want, Goal goal,
                                     Weights weight, Cut* cut) {
  S& s = smem<S>();
  if (threadIdx.x == 0) s.n_few = 0;
  __syncthreads();
  auto add = [&](float z, uint32_t id) {
    if (!(z >= weight.zlow) || coarse.bin<T>(z, weight) != h.bin) return;
    if (*(volatile uint32_t*)&s.n_few > SP_FEW) return;  // too many already
    const uint32_t at = atomicAdd(&s.n_few, 1u);
    if (at < SP_FEW) s.few[at] = ((u64)key_of<T>(z) << 32) | (uint32_t)~id;
  };
  if (S::RANKS == 1 && part.listed) {
    each_listed<T>(add);
  } else {
    uint32_t lo, hi;
    coarse.keys<T>(h.bin, weight, &lo, &hi);
    each_of_few<T, ALIGNED>(row, part, value_of<T>(lo), value_of<T>(hi), add);
  }
  __syncthreads();
  // the row's, together
  constexpr int OWN = SP_FEW / SP_THREADS;
  int n = (int)s.n_few;
  u64* few = s.row_few();
  u64 x[OWN], w[OWN];
  if constexpr (S::RANKS > 1) {
    cluster_sync();
    int from[S::RANKS + 1];
    from[0] = 0;
#pragma unroll
    for (int r = 0; r < S::RANKS; ++r) from[r + 1] = from[r] + (int)ld_cluster(&s.n_few, r);
    n = from[S::RANKS];
    if (n <= SP_FEW) {
#pragma unroll
      for (int q = 0; q < OWN; ++q) {
        const int i = threadIdx.x + q * SP_THREADS;
#pragma unroll
        for (int r = 0; r < S::RANKS; ++r) {
          if (i >= from[r] && i < from[r + 1]) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(&s.few[i - from[r]]);
            few[i] = ((u64)ld_cluster(p + 1, r) << 32) | ld_cluster(p, r);
          }
        }
      }
    }
    cluster_sync();  // the other blocks' have been read
  }
  if (n < 1 || n > SP_FEW) return false;
  sort_few<T, OWN>(few, n, weight.id_bits, s.bins[1]);
  const int i0 = OWN * threadIdx.x;
  u64 run = 0;
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    x[q] = i0 + q < n ? few[i0 + q] : 0;
    w[q] = i0 + q < n ? weight(value_of<T>((uint32_t)(x[q] >> 32))) : 0;
    run += w[q];
  }
  run = h.above_mass + mass_before(run);
  auto place = [&](int q) {
    s.found_token = x[q];
    s.found_mass = run;
    s.found_w = w[q];
  };
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    const bool yet = reached(goal, want, run, h.above + i0 + q);
    run += w[q];
    const bool now = reached(goal, want, run, h.above + i0 + q + 1);
    if ((i0 + q < n && !yet && now) || (i0 + q == n - 1 && !now)) place(q);
  }
  __syncthreads();
  *cut = {s.found_token, s.found_mass, s.found_w};
  __syncthreads();
  return true;
}

// Token and probability where thousands of tokens are equal, or nearly: a coarse bin's tokens by ranges of their keys,
// until one key is left.
template <typename T, bool ALIGNED, class S>
__device__ __noinline__ void pick_by_keys(const T* row, Share part, Coarse coarse, RowState r, Weights weight,
                                          int* token, float* prob) {
  constexpr int RANKS = S::RANKS;
  // the kept prefix: the tokens above `key` and the first `equal` of those with it, of mass `mass`
  uint32_t key = 0, equal = 0xFFFFFFFFu;
  u64 mass = r.mass, w = 0;
  if (r.top_k) {
    const Place p = descend<T, ALIGNED, S>(row, part, coarse, (u64)r.top_k, TOKENS, weight);
    key = p.key;
    equal = min((uint32_t)r.top_k - min(p.above, (uint32_t)r.top_k), p.n_equal);
    mass = p.above_mass + equal * p.w;
    w = p.w;
  }
  if (r.top_p < 1.f) {
    const u64 want = share_of(r.top_p, mass);
    const Place p = descend<T, ALIGNED, S>(row, part, coarse, want, MASS, weight);
    uint32_t j = p.n_equal;
    if (p.w && p.above_mass < want) j = (uint32_t)min((u64)j, (want - p.above_mass + p.w - 1) / p.w);
    if (p.key == key) j = min(j, equal);
    key = p.key;
    equal = j;
    mass = p.above_mass + j * p.w;
    w = p.w;
  }
  if (r.w_min > w) {
    key = 0;
    mass = mass_of_heavy<T, ALIGNED, S>(row, part, r.w_min, r.least, weight);
  }
  const u64 want = draw_at(r.u, mass);
  const Place p = descend<T, ALIGNED, S>(row, part, coarse, want, ABOVE, weight);
  uint32_t j = p.n_equal;
  if (p.w && p.above_mass <= want) j = (uint32_t)min((u64)j, (want - p.above_mass) / p.w + 1);
  if (p.key == key) j = min(j, equal);
  *token = find_token<T, ALIGNED, RANKS>(row, part, p.key, j);
  *prob = p.w ? share(p.w, mass) : 0.f;
}

// Token and probability by searches over the whole row, by one block or a cluster (ELSEWHERE in the blocks that do not
// hold the token), or over a list that holds all tokens down to the last that can be drawn.
template <typename T, bool ALIGNED, class S>
__device__ __noinline__ void pick_by_search(const T* row, Share part, RowState r, Weights weight, int* token,
                                            float* prob) {
  const Coarse coarse = {weight.far ? 0 : weight.step(weight.m), r.low, r.top, bin_shift(r.low, r.top), weight.far};
  fill_coarse<T, ALIGNED, S>(row, part, coarse, weight, r.top_k != 0);
  // each filter's last token: its place in the bins, then among its bin's tokens
  Cut cut = {0, r.mass, 0};
  auto search = [&](u64 want, Goal goal) {
    return resolve<T, ALIGNED, S>(row, part, coarse, find_bin<S>(0, 0, 0, want, goal), want, goal, weight, &cut);
  };
  bool found = !r.top_k || search((u64)r.top_k, TOKENS);
  if (found && r.top_p < 1.f) found = search(share_of(r.top_p, cut.mass), MASS);
  if (found) {
    // min-p alone (the mass is not known yet), or above what top-k and top-p keep
    u64 mass = cut.mass;
    if (r.w_min > cut.w) mass = mass_of_heavy<T, ALIGNED, S>(row, part, r.w_min, r.least, weight);
    found = search(draw_at(r.u, mass), ABOVE);
    if (found) {
      *token = S::RANKS == 1 || cluster_rank() == 0 ? (int)~(uint32_t)cut.token : ELSEWHERE;
      *prob = share(cut.w, mass);
      return;
    }
  }
  if (S::RANKS == 1 && part.listed) {
    part.listed = false;
    fill_coarse<T, ALIGNED, S>(row, part, coarse, weight, r.top_k != 0);
  }
  pick_by_keys<T, ALIGNED, S>(row, part, coarse, r, weight, token, prob);
}

// f(maximum, group) of every group, eight to a thread in flight.
template <typename F>
__device__ __forceinline__ void each_group(const float* gmax, int n_groups, F f) {
  static_assert(SEG_GROUPS % 4 == 0, "whole vectors");
  const float4* v = reinterpret_cast<const float4*>(gmax);
  for (int i = threadIdx.x; 4 * i < n_groups; i += 2 * SP_THREADS) {
    const bool two = 4 * (i + SP_THREADS) < n_groups;
    const float4 x = v[i];
    float4 y;
    if (two) y = v[i + SP_THREADS];
    f(x.x, 4 * i);
    f(x.y, 4 * i + 1);
    f(x.z, 4 * i + 2);
    f(x.w, 4 * i + 3);
    if (two) {
      const int j = i + SP_THREADS;
      f(y.x, 4 * j);
      f(y.y, 4 * j + 1);
      f(y.z, 4 * j + 2);
      f(y.w, 4 * j + 3);
    }
  }
}

// The lower edge of the histogram bin that holds the k-th largest of the groups' maxima (of the list, without them),
// of which the smallest above -inf has the key lo: at least k tokens reach it.  0 where fewer than k are above -inf.
template <typename T>
__device__ __noinline__ uint32_t bound_by_count(const float* gmax, int n_groups, uint32_t lo,
                                                uint32_t top, uint32_t k) {
  SampleSmem& s = smem<SampleSmem>();
  constexpr int OWN = SP_BINS / SP_THREADS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sh = bin_shift(lo, top);
  for (int b = threadIdx.x; b < SP_BINS; b += SP_THREADS) s.group_count[b] = 0;
  if (threadIdx.x == 0) s.bin = -1;
  __syncthreads();
  if (gmax) {
    each_group(gmax, n_groups, [&](float z, int) {
      const uint32_t x = key_of<T>(z);
      if (x >= lo) atomicAdd(&s.group_count[(top - x) >> sh], 1u);
    });
  } else {
    for (int i = threadIdx.x; i < (int)s.n_list; i += SP_THREADS)
      atomicAdd(&s.group_count[(top - (uint32_t)(s.list[i] >> 32)) >> sh], 1u);
  }
  __syncthreads();
  uint32_t c = 0;
  const int b0 = threadIdx.x * OWN;
#pragma unroll
  for (int q = 0; q < OWN; ++q) c += s.group_count[b0 + q];
  uint32_t inc = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s.warp_count[warp] = inc;
  __syncthreads();
  uint32_t at = inc - c;
  for (int w = 0; w < warp; ++w) at += s.warp_count[w];
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    if (at < k && at + s.group_count[b0 + q] >= k) s.bin = b0 + q;
    at += s.group_count[b0 + q];
  }
  __syncthreads();
  const int b = s.bin;
  __syncthreads();
  if (b < 0) return 0;
  const uint32_t hi = top - ((uint32_t)b << sh), reach = (1u << sh) - 1u;
  return hi - lo > reach ? hi - reach : lo;
}

// Lists the tokens whose keys reach `lo`, from the groups whose maxima do; false where they are too many.
template <typename T, bool ALIGNED>
__device__ __noinline__ bool list_tokens(const T* row, int vocab, const float* gmax, int n_groups,
                                         uint32_t lo) {
  SampleSmem& s = smem<SampleSmem>();
  constexpr int PER = Elem<T>::PER16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s.n_list = s.n_groups = 0;
  __syncthreads();
  const float from = value_of<T>(lo);
  each_group(gmax, n_groups, [&](float z, int g) {
    if (z >= from) {
      const uint32_t at = atomicAdd(&s.n_groups, 1u);
      if (at < SP_GROUPS) s.groups[at] = g;
    }
  });
  __syncthreads();
  const uint32_t n = s.n_groups;
  if (n > SP_GROUPS) return false;
  // two groups to a warp, 16 vectors each, the loads of AHEAD pairs of groups in flight (registers for no more)
  constexpr int AHEAD = 4;
  const Within<T> within(from, INFINITY);  // (a row with +inf does not come here)
  for (uint32_t i0 = warp * 2; i0 < n; i0 += SP_WARPS * 2 * AHEAD) {
    uint4 u[AHEAD];
    uint32_t id[AHEAD], hits[AHEAD], inc = 0;
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const uint32_t i = i0 + q * SP_WARPS * 2 + (lane >> 4);
      id[q] = (uint32_t)vocab;
      if (i < n) {
        const uint32_t g = s.groups[i];
        id[q] = (g / SEG_GROUPS) * row_seg<T>() + (((lane >> 2) & 3) * 32 + (g % SEG_GROUPS) * 4 + (lane & 3)) * PER;
      }
      if ((int)id[q] < vocab) u[q] = row_vec<T, ALIGNED>(row, (int)id[q], vocab);
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      hits[q] = (int)id[q] < vocab ? within(u[q]) : 0u;
      inc += __popc(hits[q]);
    }
    const uint32_t own = inc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    uint32_t at = 0;
    if (lane == 31 && inc) at = atomicAdd(&s.n_list, inc);
    at = __shfl_sync(0xFFFFFFFFu, at, 31) + inc - own;
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      for (uint32_t h = hits[q]; h; h &= h - 1, ++at) {
        const int e = __ffs(h) - 1;
        if (at < SP_LIST) s.list[at] = ((u64)key_of<T>(element<T>(u[q], e)) << 32) | (uint32_t)~(id[q] + e);
      }
    }
  }
  __syncthreads();
  return s.n_list <= SP_LIST;
}

// Leaves those of the list whose keys reach `lo`.
__device__ __noinline__ void shorten_list(uint32_t lo) {
  SampleSmem& s = smem<SampleSmem>();
  constexpr int OWN = SP_LIST / SP_THREADS;
  u64 x[OWN];
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    const int i = threadIdx.x + q * SP_THREADS;
    x[q] = i < (int)s.n_list ? s.list[i] : 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) s.n_list = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < OWN; ++q)
    if (x[q] && (uint32_t)(x[q] >> 32) >= lo) s.list[atomicAdd(&s.n_list, 1u)] = x[q];
  __syncthreads();
}

// The mass of the list.
template <typename T>
__device__ __noinline__ u64 list_mass(Weights weight) {
  SampleSmem& s = smem<SampleSmem>();
  u64 sum = 0;
  for (int i = threadIdx.x; i < (int)s.n_list; i += SP_THREADS) sum += weight(value_of<T>((uint32_t)(s.list[i] >> 32)));
  return block_mass(sum);
}

// Token and probability from a list of at most SP_SORT tokens, sorted here, which holds all tokens down to the last
// that can be drawn; OWN to a thread.
template <typename T, int OWN>
__device__ __noinline__ void pick_from_list(RowState r, Weights weight, int* token, float* prob) {
  SampleSmem& s = smem<SampleSmem>();
  const int n = (int)s.n_list, i0 = OWN * threadIdx.x;
  sort_few<T, OWN>(s.list, n, weight.id_bits, s.bins[1]);
  u64 run[OWN + 1];  // the sums up to each token
  run[0] = 0;
  int heavy = 0;
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    const u64 w = i0 + q < n ? weight(value_of<T>((uint32_t)(s.list[i0 + q] >> 32))) : 0;
    heavy += i0 + q < n && w >= r.w_min;
    run[q + 1] = run[q] + w;
  }
  if (threadIdx.x == 0) {
    s.found_mass = r.mass;
    s.found_at = n;
    s.n_few = 0;  // of the tokens that min-p keeps
  }
  const u64 before = mass_before(run[OWN]);  // (a barrier inside)
#pragma unroll
  for (int q = 0; q <= OWN; ++q) run[q] += before;
  if (r.w_min) {
    heavy = __reduce_add_sync(0xFFFFFFFFu, heavy);
    if ((threadIdx.x & 31) == 0 && heavy) atomicAdd(&s.n_few, (unsigned)heavy);
  }
  // the mass up to and with the last token that is kept
  int keep = n;
  u64 mass = r.mass;
  auto mass_of_kept = [&]() {
#pragma unroll
    for (int q = 0; q < OWN; ++q)
      if (i0 + q == keep - 1) s.found_mass = run[q + 1];
    __syncthreads();
    mass = s.found_mass;
  };
  if (r.top_k) {
    keep = min(n, r.top_k);
    mass_of_kept();
  }
  if (r.top_p < 1.f) {
    const u64 want = share_of(r.top_p, mass);
#pragma unroll
    for (int q = 0; q < OWN; ++q)
      if (i0 + q < n && run[q] < want && run[q + 1] >= want) s.found_at = i0 + q + 1;
  }
  __syncthreads();
  keep = min(keep, (int)s.found_at);
  if (r.w_min) keep = min(keep, max(1, (int)s.n_few));
  if (r.top_p < 1.f || r.w_min) mass_of_kept();
  const u64 want = draw_at(r.u, mass);
  // the last kept one where rounding leaves no other
#pragma unroll
  for (int q = 0; q < OWN; ++q) {
    const int i = i0 + q;
    if (i < n && i < keep && run[q] <= want && (run[q + 1] > want || i == keep - 1)) {
      s.found_id = ~(uint32_t)s.list[i];
      s.found_w = run[q + 1] - run[q];
    }
  }
  __syncthreads();
  *token = (int)s.found_id;
  *prob = share(s.found_w, mass);
}

// A row that is searched by k_sample_search.
struct Job {
  RowState row;
  float m;
  int searched;
};

template <typename T, bool ALIGNED, bool SHORT>
__global__ void __launch_bounds__(SP_THREADS, 2) k_sample_pick(SampleArgs a, int n_seg, const float* gmax_all,
                                                               const SegMass* segs_all, Job* jobs) {
  SampleSmem& s = smem<SampleSmem>();
  __shared__ __align__(16) float s_gmax[SHORT ? SP_WARPS * SEG_GROUPS : 1];
  __shared__ SegMass s_seg[SHORT ? SP_WARPS : 1];
  const int n = blockIdx.x, vocab = a.vocab, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < (int)(sizeof(ExpTable) / 4); i += SP_THREADS)
    reinterpret_cast<uint32_t*>(&s.tab)[i] = reinterpret_cast<const uint32_t*>(&g_exp_table)[i];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!SHORT && jobs) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the searching kernel follows
  const T* row = static_cast<const T*>(a.logits) + n * a.ld;
  const float t = a.temperature ? __ldg(a.temperature + n) : a.temperature0;
  const float top_p = a.top_p ? __ldg(a.top_p + n) : a.top_p0, min_p = a.min_p ? __ldg(a.min_p + n) : a.min_p0;
  const int top_k = a.top_k ? __ldg(a.top_k + n) : a.top_k0;
  const float u = __ldg(a.u + n);
  const bool whole = needs_mass(t, top_k, top_p, min_p, vocab);
  const float* gmax = gmax_all + (long long)n * n_seg * SEG_GROUPS;
  const SegMass* segs = segs_all + (long long)n * n_seg;
  if constexpr (SHORT) {
    ScanTable& table = *reinterpret_cast<ScanTable*>(s.list);  // (not used before)
    if (whole) {
      fill_table(table, SP_THREADS);
      __syncthreads();
    }
    if (warp < n_seg) scan_segment<T, ALIGNED>(row, warp, vocab, t, whole, table, s_gmax, s_seg);
    gmax = s_gmax;
    segs = s_seg;
    __syncthreads();
  }
  const int n_groups = n_seg * SEG_GROUPS;
  // the row's largest logit, and the smallest of the groups' maxima above -inf
  float m = -INFINITY, least_max = INFINITY;
  each_group(gmax, n_groups, [&](float x, int) {
    m = max_nan(m, x);
    if (x > -INFINITY) least_max = fminf(least_max, x);
  });
  m = warp_max(m);
  for (int o = 16; o > 0; o >>= 1) least_max = fminf(least_max, __shfl_xor_sync(0xFFFFFFFFu, least_max, o));
  if (lane == 0) {
    s.warp_max[warp] = m;
    s.warp_min[warp] = least_max;
  }
  __syncthreads();
  for (int w = 0; w < SP_WARPS; ++w) {
    m = max_nan(m, s.warp_max[w]);
    least_max = fminf(least_max, s.warp_min[w]);
  }
  __syncthreads();
  int token = -1;
  float prob = 0.f;
  bool searched = false;
  // no distribution: a NaN or +inf logit, nothing above -inf, settings or uniforms that are not numbers
  if (fabsf(m) < INFINITY && t >= 0.f && t < INFINITY && top_p == top_p && min_p == min_p && u == u) {
    RowState r;
    r.top = key_of<T>(m);
    if (t == 0.f || top_k == 1 || top_p <= 0.f) {
      if (list_tokens<T, ALIGNED>(row, vocab, gmax, n_groups, r.top)) {
        // the lowest of the ids that share the largest logit
        uint32_t id = 0xFFFFFFFFu;
        for (int i = threadIdx.x; i < (int)s.n_list; i += SP_THREADS) id = min(id, ~(uint32_t)s.list[i]);
        id = __reduce_min_sync(0xFFFFFFFFu, id);
        if (lane == 0) s.warp_count[warp] = id;
        __syncthreads();
        for (int w = 0; w < SP_WARPS; ++w) id = min(id, s.warp_count[w]);
        token = (int)id;
      } else {
        __syncthreads();
        token = find_token<T, ALIGNED, 1>(row, Share{0, vocab, false}, r.top, 1);
      }
      prob = 1.f;
    } else {
      const Weights weight(m, t, vocab);
      r.low = key_of<T>(weight.zlow);
      // (the limit itself need not be a value of T: the key is then that of the value below)
      if (value_of<T>(r.low) < weight.zlow) ++r.low;
      r.top_k = top_k > 1 && top_k < vocab ? top_k : 0;
      r.top_p = top_p;
      r.u = u;
      r.mass = 0;
      r.least = 0;
      r.w_min = 0;
      if (min_p > 0.f) {
        const u64 most = weight(m);
        bool rest;
        r.w_min = min_p < 1.f ? times(min_p, most, &rest) : most;
        if (min_p < 1.f) r.w_min += rest;
        // a little lower: this value's and the weights' roundings
        const float z = m + t * logf(fminf(min_p, 1.f));
        r.least = min(key_of<T>(z - 1e-5f * (fabsf(z) + fabsf(m)) - 1e-3f * t), r.top);
      }
      if (whole || (!r.top_k && r.top_p < 1.f)) {
        u64 sum = 0;
        if (weight.far) {
          each<T, ALIGNED>(row, Share{0, vocab, false}, weight.zlow, weight.m, [&](float z) { sum += weight(z); });
        } else {
          for (int i = threadIdx.x; i < n_seg; i += SP_THREADS) {
            const SegMass q = segs[i];
            const long long down = (long long)(SEG_FRAC - weight.frac) + weight.e_ref - q.e;
            if (down <= 0) sum += q.mass;
            else if (down < 64) sum += (q.mass + (1ull << (down - 1))) >> down;
          }
        }
        r.mass = block_mass(sum);
      }
      // a list of the tokens from a key on below which nothing can be kept and drawn
      bool listed = false;
      if (whole) {
        // the mass that the list has to hold
        const u64 want = r.top_p < 1.f ? share_of(r.top_p, r.mass) : draw_at(r.u, r.mass) + 1;
        const uint32_t lo =
            SP_TRY < n_groups ? bound_by_count<T>(gmax, n_groups, key_of<T>(least_max), r.top, SP_TRY) : 0;
        if (list_tokens<T, ALIGNED>(row, vocab, gmax, n_groups, max(lo, r.low)))
          listed = lo <= r.low || list_mass<T>(weight) >= want;
      } else {
        uint32_t lo = r.top_k ? 0 : r.least;
        if (r.top_k && r.top_k <= n_groups)
          lo = bound_by_count<T>(gmax, n_groups, key_of<T>(least_max), r.top, (uint32_t)r.top_k);
        lo = max(lo, r.low);
        listed = list_tokens<T, ALIGNED>(row, vocab, gmax, n_groups, lo);
        // more tokens than are sorted: only the first top_k of them count (512 rows of top-k 1000: 92 us searched)
        if (listed && s.n_list > SP_SORT && r.top_k && r.top_k < SP_SORT)
          shorten_list(bound_by_count<T>(nullptr, 0, lo, r.top, (uint32_t)r.top_k));
      }
      if (listed && s.n_list <= SP_SORT) {
        // (a token to a thread where that does: 512 rows of 50 tokens 46 us, 48 with four)
        if (s.n_list <= SP_THREADS) pick_from_list<T, 1>(r, weight, &token, &prob);
        else pick_from_list<T, SP_SORT / SP_THREADS>(r, weight, &token, &prob);
      } else if (listed) {
        pick_by_search<T, ALIGNED, SampleSmem>(row, Share{0, vocab, true}, r, weight, &token, &prob);
      } else if (SHORT || !jobs) {
        __syncthreads();
        pick_by_search<T, ALIGNED, SampleSmem>(row, Share{0, vocab, false}, r, weight, &token, &prob);
      } else {
        // left to k_sample_search
        if (threadIdx.x == 0) jobs[n].row = r;
        searched = true;
      }
    }
  }
  if (!SHORT && jobs && threadIdx.x == 0) {
    jobs[n].m = m;
    jobs[n].searched = searched;
  }
  if (searched) return;
  if (threadIdx.x == 0) {
    a.token[n] = token;
    if (a.prob) a.prob[n] = prob;
  }
}

// The rows whose lists would have been too long, each by a cluster.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(SP_THREADS, 2) k_sample_search(SampleArgs a, const Job* jobs) {
  SearchSmem& s = smem<SearchSmem>();
  const int n = blockIdx.x / SS_RANKS;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!__ldcg(&jobs[n].searched)) return;  // the whole cluster
  for (int i = threadIdx.x; i < (int)(sizeof(ExpTable) / 4); i += SP_THREADS)
    reinterpret_cast<uint32_t*>(&s.tab)[i] = reinterpret_cast<const uint32_t*>(&g_exp_table)[i];
  __syncthreads();
  const RowState r = jobs[n].row;
  const float t = a.temperature ? __ldg(a.temperature + n) : a.temperature0;
  const Weights weight(jobs[n].m, t, a.vocab);
  int token;
  float prob;
  pick_by_search<T, ALIGNED, SearchSmem>(static_cast<const T*>(a.logits) + n * a.ld,
                                         share_of_row<T, SS_RANKS>(a.vocab), r, weight, &token, &prob);
  if (threadIdx.x == 0 && token != ELSEWHERE) {
    a.token[n] = token;
    if (a.prob) a.prob[n] = prob;
  }
}

}  // namespace

namespace {

struct SampleLayout {
  size_t gmax, segs, jobs, total;
  int n_seg;
};
SampleLayout sample_layout(int N, int vocab, int dtype) {
  const int seg = dtype == DH_BF16 ? row_seg<__nv_bfloat16>() : row_seg<float>();
  SampleLayout L;
  L.n_seg = (vocab + seg - 1) / seg;
  L.gmax = WS_HEADER;
  L.segs = L.gmax + align_up((size_t)N * L.n_seg * SEG_GROUPS * sizeof(float), 256);
  L.jobs = L.segs + align_up((size_t)N * L.n_seg * sizeof(SegMass), 256);
  L.total = L.n_seg <= SP_WARPS ? 0 : L.jobs + align_up((size_t)N * sizeof(Job), 256);
  return L;
}

// Rows that the host knows to have a small top-k, or temperature 0: their lists are too long only where thousands of
// tokens are equal, and then the block that picks searches too.  A third kernel would cost the usual call 2 us.
bool seldom_searched(const SampleArgs& a) {
  return (!a.temperature && a.temperature0 == 0.f) ||
         (!a.top_k && a.top_k0 >= 1 && a.top_k0 <= 1024 && a.top_k0 < a.vocab);
}

template <typename T, bool ALIGNED>
cudaError_t run_sample(const Ctx& c, const SampleArgs& a, int dtype) {
  const SampleLayout L = sample_layout(a.N, a.vocab, dtype);
  const dim3 grid((unsigned)a.N), block(SP_THREADS);
  const size_t smem = sizeof(SampleSmem);
  if (L.total == 0) {
    static unsigned long long short_done = 0;
    const cudaError_t e = allow_max_smem(k_sample_pick<T, ALIGNED, true>, c.device, &short_done);
    if (e != cudaSuccess) return e;
    return launch_pdl(c, "sample_pick", k_sample_pick<T, ALIGNED, true>, grid, block, smem, a, L.n_seg, nullptr,
                      nullptr, nullptr);
  }
  static unsigned long long long_done = 0;
  cudaError_t e = allow_max_smem(k_sample_pick<T, ALIGNED, false>, c.device, &long_done);
  if (e != cudaSuccess) return e;
  float* gmax = reinterpret_cast<float*>(static_cast<char*>(a.ws) + L.gmax);
  SegMass* segs = reinterpret_cast<SegMass*>(static_cast<char*>(a.ws) + L.segs);
  const long long want = ((long long)a.N * L.n_seg + SC_THREADS / 32 - 1) / (SC_THREADS / 32);
  const long long most = (long long)SC_BLOCKS * c.num_sms;
  e = launch_pdl(c, "sample_scan", k_sample_scan<T, ALIGNED>, dim3((unsigned)(want < most ? want : most)),
                 dim3(SC_THREADS), 0, a, L.n_seg, gmax, segs);
  if (e != cudaSuccess) return e;
  Job* jobs = seldom_searched(a) ? nullptr : reinterpret_cast<Job*>(static_cast<char*>(a.ws) + L.jobs);
  e = launch_pdl(c, "sample_pick", k_sample_pick<T, ALIGNED, false>, grid, block, smem, a, L.n_seg, gmax, segs, jobs);
  if (e != cudaSuccess || !jobs) return e;
  static unsigned long long search_done = 0;
  e = allow_max_smem(k_sample_search<T, ALIGNED>, c.device, &search_done);
  if (e != cudaSuccess) return e;
  return launch_clusters(c, "sample_search", k_sample_search<T, ALIGNED>, SS_RANKS, dim3((unsigned)a.N * SS_RANKS),
                         block, sizeof(SearchSmem), a, jobs);
}

}  // namespace

size_t sample_workspace(int N, int vocab, int dtype) { return sample_layout(N, vocab, dtype).total; }

cudaError_t launch_sample(const Ctx& c, const SampleArgs& a, int dtype) {
  const int elem = dtype == DH_BF16 ? 2 : 4;
  const bool al = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && (a.N == 1 || a.ld * elem % 16 == 0);
  if (dtype == DH_BF16)
    return al ? run_sample<__nv_bfloat16, true>(c, a, dtype) : run_sample<__nv_bfloat16, false>(c, a, dtype);
  return al ? run_sample<float, true>(c, a, dtype) : run_sample<float, false>(c, a, dtype);
}

}  // namespace dh
