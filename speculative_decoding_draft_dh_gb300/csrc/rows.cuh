// Rows of vocabulary logits, shared by the operators that reduce them (distill.cu, beam.cu).
//
// A row has `vocab` logits of type T at any element-aligned address (rows may be strided and a
// vocabulary need not be a multiple of anything).  A vector is 16 bytes of elements counted from
// the row's first one, so which elements a lane holds, and with it the order of every sum, depends
// on the position in the row alone, not on the row's address: equal rows give equal sums.
#pragma once

#include "operators.cuh"

namespace dh {

// 2^x on the special-function unit, subnormal results flushed to zero (the terms it flushes are
// below 2^-126 of the largest term's and do not move a sum).
__device__ __forceinline__ float row_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float ROW_LOG2E = 1.4426950408889634f;

// The 16 bytes at an address of any alignment s = address mod 16, taken from the one or two aligned
// 16-byte words that hold them (both hold bytes of the vector, so neither lies outside the row's
// memory by a whole word).
__device__ __forceinline__ uint4 ld16_any(const void* p) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  const unsigned s = (unsigned)a & 15u;
  const uint4* w = reinterpret_cast<const uint4*>(a - s);
  const uint4 lo = __ldg(w);
  if (s == 0) return lo;
  const uint4 hi = __ldg(w + 1);
  // words q .. q + 4 of the eight, then a shift by the bytes within a word
  const unsigned q = s >> 2, b = (s & 3u) * 8u;
  uint32_t x0, x1, x2, x3, x4;
  if (q == 0) { x0 = lo.x; x1 = lo.y; x2 = lo.z; x3 = lo.w; x4 = hi.x; }
  else if (q == 1) { x0 = lo.y; x1 = lo.z; x2 = lo.w; x3 = hi.x; x4 = hi.y; }
  else if (q == 2) { x0 = lo.z; x1 = lo.w; x2 = hi.x; x3 = hi.y; x4 = hi.z; }
  else { x0 = lo.w; x1 = hi.x; x2 = hi.y; x3 = hi.z; x4 = hi.w; }
  return make_uint4(__funnelshift_r(x0, x1, b), __funnelshift_r(x1, x2, b), __funnelshift_r(x2, x3, b),
                    __funnelshift_r(x3, x4, b));
}

// Two elements of type T equal to -inf, as a 32-bit word (fp32: one element).
template <typename T> struct NegInf;
template <> struct NegInf<float> { static constexpr uint32_t WORD = 0xFF800000u; };
template <> struct NegInf<__nv_bfloat16> { static constexpr uint32_t WORD = 0xFF80FF80u; };

__device__ __forceinline__ uint32_t elem_bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t elem_bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }

// Elements id .. id + PER16 - 1 of a row, -inf past its end: the row's last, partial vector.
template <typename T>
__device__ __forceinline__ uint4 row_tail(const T* row, int id, int vocab) {
  constexpr int PER = Elem<T>::PER16;
  uint32_t w[4] = {NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD};
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    if (id + e < vocab) {
      const uint32_t b = elem_bits(row[id + e]);
      if (sizeof(T) == 4) w[e] = b;
      else w[e / 2] = (e & 1) ? ((w[e / 2] & 0xFFFFu) | (b << 16)) : ((w[e / 2] & 0xFFFF0000u) | b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __noinline__ uint4 row_tail_call(const T* row, int id, int vocab) { return row_tail<T>(row, id, vocab); }
template <typename T>
__device__ __noinline__ uint4 ld16_any_call(const T* p) { return ld16_any(p); }

// Elements id .. id + PER16 - 1 of a row, -inf past its end.  ALIGNED: the row starts on 16 bytes.
// SMALL: the rare paths are calls, for code that is run once and unrolled (its instructions come from
// memory).
template <typename T, bool ALIGNED, bool SMALL = false>
__device__ __forceinline__ uint4 row_vec(const T* row, int id, int vocab) {
  if (id + Elem<T>::PER16 <= vocab)
    return ALIGNED ? ld_nc_v4(row + id) : (SMALL ? ld16_any_call<T>(row + id) : ld16_any(row + id));
  return SMALL ? row_tail_call<T>(row, id, vocab) : row_tail<T>(row, id, vocab);
}

// Maximum that a NaN passes through, so that a row which holds one is found out.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Largest element of N vectors, NaN if there is one.
template <typename T, int N>
__device__ __forceinline__ float vec_max(const uint4 (&u)[N]) {
  if constexpr (sizeof(T) == 4) {
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < N; ++v)
      m = max_nan(m, max_nan(max_nan(__uint_as_float(u[v].x), __uint_as_float(u[v].y)),
                             max_nan(__uint_as_float(u[v].z), __uint_as_float(u[v].w))));
    return m;
  } else {
    // pairwise in bf16: the maximum of bf16 values is one of them, so nothing is rounded
    auto b2 = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    __nv_bfloat162 m = b2(NegInf<T>::WORD);
#pragma unroll
    for (int v = 0; v < N; ++v)
      m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(b2(u[v].x), b2(u[v].y)), __hmax2_nan(b2(u[v].z), b2(u[v].w))));
    return max_nan(__low2float(m), __high2float(m));
  }
}

// Two fp32 operations in one instruction, each rounded as its scalar form, on a pair in one register
// pair.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The reference of a row's exponentials, in powers of two: 2^(z c - r) with r the rounded m c, so a
// term takes one fused multiply-add and its argument one rounding.  What r's rounding leaves out,
// m c - r, is the same factor for every term: excess() gives it to those who want the sum relative
// to exp(z/T - m/T).  It is below 2^-15 in the exponent while |m c| < 1024; beyond that (large logits,
// small temperatures, the type's limits) `far` asks for the terms by (z - m) c instead.
struct ExpRef {
  float m, r;
  bool far;
  __device__ __forceinline__ ExpRef(float m_, float c) : m(m_), r(m_ * c), far(!(fabsf(m_ * c) < 1024.f)) {
    if (far) r = 0.f;
  }
  // sum 2^((z - m) c) from sum 2^(z c - r): 2^-x for the small x = m c - r by its first two terms
  __device__ __forceinline__ float by_max(float s, float c) const {
    return far ? s : fmaf(s, -0.6931471805599453f * fmaf(m, c, -r), s);
  }
};

// The exponentials of the elements of a vector, in pairs.
template <typename T>
__device__ __forceinline__ void vec_exp(const uint4& u, const ExpRef& e, float c, f32x2* z) {
  constexpr int PER = Elem<T>::PER16;
  float x[PER];
  Elem<T>::unpack(u, x);
  if (__builtin_expect(e.far, 0)) {
#pragma unroll
    for (int q = 0; q < PER; ++q) x[q] = (x[q] - e.m) * c;
  } else {
    const f32x2 cc = pack2(c, c), nr = pack2(-e.r, -e.r);
#pragma unroll
    for (int q = 0; q < PER / 2; ++q) unpack2(fma2(pack2(x[2 * q], x[2 * q + 1]), cc, nr), x[2 * q], x[2 * q + 1]);
  }
#pragma unroll
  for (int q = 0; q < PER / 2; ++q) z[q] = pack2(row_ex2(x[2 * q]), row_ex2(x[2 * q + 1]));
}
__device__ __forceinline__ float one_exp(float z, const ExpRef& e, float c) {
  return row_ex2(e.far ? (z - e.m) * c : fmaf(z, c, -e.r));
}

// Their sum, in a fixed tree.
template <typename T>
__device__ __forceinline__ float vec_expsum(const uint4& u, const ExpRef& e, float c) {
  f32x2 z[Elem<T>::PER16 / 2];
  vec_exp<T>(u, e, c, z);
  f32x2 s = add2(z[0], z[1]);
  if constexpr (Elem<T>::PER16 == 8) s = add2(s, add2(z[2], z[3]));
  float a, b;
  unpack2(s, a, b);
  return a + b;
}

// The elements of a vector, each rounded once to the logits' type.
template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float* z) {
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

// a times the exponentials of a vector's elements, rounded once to the logits' type.
template <typename T>
__device__ __forceinline__ uint4 grad_vec(const uint4& u, const ExpRef& e, float c, float a) {
  f32x2 z[Elem<T>::PER16 / 2];
  vec_exp<T>(u, e, c, z);
  const f32x2 aa = pack2(a, a);
  float x[Elem<T>::PER16];
#pragma unroll
  for (int q = 0; q < Elem<T>::PER16 / 2; ++q) unpack2(mul2(z[q], aa), x[2 * q], x[2 * q + 1]);
  return pack_vec<T>(x);
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// row_vec for memory that the kernel may write later (no read-only loads); any alignment.
template <typename T>
__device__ __forceinline__ uint4 row_vec_rw(const T* row, int id, int vocab) {
  constexpr int PER = Elem<T>::PER16;
  uint4 r;
  if (id + PER <= vocab && (reinterpret_cast<uintptr_t>(row + id) & 15u) == 0) {
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(row + id) : "memory");
    return r;
  }
  uint32_t w[4] = {NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD, NegInf<T>::WORD};
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    if (id + e < vocab) {
      if constexpr (sizeof(T) == 4) {
        w[e] = __float_as_uint(*(const volatile float*)(row + id + e));
      } else {
        const uint32_t b = *(const volatile unsigned short*)(row + id + e);
        w[e / 2] = (e & 1) ? ((w[e / 2] & 0xFFFFu) | (b << 16)) : ((w[e / 2] & 0xFFFF0000u) | b);
      }
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Segments of a row: ROW_SEG_VECS vectors per lane of one warp (1024 bf16 or 512 fp32 ids), lane l
// holding vectors l, l + 32, ...  k_row_stats leaves each segment's (max, sum of exp((z - max)/T)).
constexpr int ROW_SEG_VECS = 4;
template <typename T> constexpr int row_seg() { return 32 * Elem<T>::PER16 * ROW_SEG_VECS; }

// A segment's pair from its vectors, by one warp (every lane gets it).
template <typename T>
__device__ __forceinline__ float2 segment_stats(const uint4 (&u)[ROW_SEG_VECS], float c) {
  const float m = warp_max(vec_max<T>(u));
  float s = 0.f;
  if (m != -INFINITY) {
    const ExpRef ref(m, c);
    float p[ROW_SEG_VECS];
#pragma unroll
    for (int v = 0; v < ROW_SEG_VECS; ++v) p[v] = vec_expsum<T>(u[v], ref, c);
    s = ref.by_max(warp_sum((p[0] + p[1]) + (p[2] + p[3])), c);
  }
  return make_float2(m, s);
}

// A sum of positive terms held as a rounded value and the part that rounding left out (the
// two-term sum of Knuth): combining the segments' sums in any number adds no error that counts.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
  }
};

// log(hi + lo) of a positive sum in two floats, as two floats, to about 3e-9: 64-bit operations keep
// an SM's one slow unit for 16 cycles each (a 64-bit logarithm took 2,600 cycles where this takes 300).
// With hi = 2^k f, f in [2/3, 4/3), and t = (f - 1)/(f + 1), log f = 2 artanh t
// = 2 t + 2 t (t^2/3 + t^4/5 + ...): the first term in two floats, the rest, below 0.02 t, in one.
__device__ __forceinline__ Sum2 log_sum(float hi, float lo) {
  int k = (int)((__float_as_uint(hi) + 0x00555555u) >> 23) - 127;  // rounds to the nearest in [2/3, 4/3)
  const float scale = __uint_as_float((uint32_t)(127 - k) << 23);
  const float f = hi * scale, fl = lo * scale;  // exact
  const float a = f - 1.f;                      // exact; the numerator is a + fl
  const float b = f + 1.f, bl = (f - (b - 1.f)) + fl;
  const float t = a / b;
  const float tl = ((fmaf(-t, b, a) + fl) - t * bl) / b;
  const float q = t * t;
  const float r = q * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 1.f / 11.f, 1.f / 9.f), 1.f / 7.f), 1.f / 5.f), 1.f / 3.f);
  Sum2 s;
  // log 2 as 355/512, whose product with k is exact, and the rest (the split of Cody and Waite)
  s.add((float)k * 0.693359375f);
  s.add(2.f * t);
  s.lo += (float)k * -2.12194440e-4f + 2.f * (tl + t * r);
  return s;
}

// A row's (max, sum) from its segments' pairs, by one warp; every lane gets the result.  The sum
// is relative to exp((z - max)/T); a row of -inf gives (-inf, 0).  A NaN logit gives
// (NaN, NaN), a +inf one (+inf, NaN).  inv_t = 1 / T.
// maxima (may be null): takes the segments' maxima.
__device__ __forceinline__ void row_combine(const float2* seg, int n_seg, float inv_t, float* m_out,
                                            Sum2* sum_out, float* maxima = nullptr) {
  constexpr int HELD = 8;  // pairs per lane that stay in registers, their loads in flight together
  const int lane = threadIdx.x & 31;
  float2 q[HELD];
  float m = -INFINITY;
#pragma unroll
  for (int e = 0; e < HELD; ++e)
    q[e] = lane + e * 32 < n_seg ? seg[lane + e * 32] : make_float2(-INFINITY, 0.f);
#pragma unroll
  for (int e = 0; e < HELD; ++e) {
    m = max_nan(m, q[e].x);
    if (maxima && lane + e * 32 < n_seg) maxima[lane + e * 32] = q[e].x;
  }
  for (int i = lane + HELD * 32; i < n_seg; i += 32) {
    const float x = seg[i].x;
    m = max_nan(m, x);
    if (maxima) maxima[i] = x;
  }
  m = warp_max(m);
  Sum2 s;
  // a segment of -inf alone adds nothing; a NaN sum stays one
  auto add = [&](const float2& p) {
    if (p.x != -INFINITY) s.add(p.y * expf((p.x - m) * inv_t));
  };
#pragma unroll
  for (int e = 0; e < HELD; ++e) add(q[e]);
  for (int i = lane + HELD * 32; i < n_seg; i += 32) add(seg[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xFFFFFFFFu, s.hi, o), l = __shfl_xor_sync(0xFFFFFFFFu, s.lo, o);
    // the lower lane's first, so that both lanes compute the same
    Sum2 a = (threadIdx.x & o) ? Sum2{h, l} : s;
    const Sum2 b = (threadIdx.x & o) ? s : Sum2{h, l};
    a.add(b.hi);
    a.lo += b.lo;
    s = a;
  }
  *m_out = m;
  *sum_out = s;
}

}  // namespace dh
