// Distillation, statistics and dense gradient in one pass over the logits (definitions at
// dh_distill_topk in dh.h; distill.cu has the other kernels).
//
// The gradient g T (q - p) needs the row's normaliser, so a row is read to its end before its first
// gradient can be written.  Here a row stays in the shared memory of a cluster of C CTAs from its one
// read to its one write: 4 bytes of traffic per bf16 logit instead of the 6 of two passes.
//
// k_distill_ring: persistent clusters, each walking rows; CTA c holds the c-th slice.
//   producer (one thread)   bulk-copies the slices, chunk by chunk and row after row, into a ring of
//                           slots; it runs ahead of the row at work by what the ring holds beyond a
//                           slice, so memory stays busy through the reductions.
//   consumers (20 warps)    pass A: maximum and sum of exp of the chunks as they arrive, each thread
//                           with a running maximum; every warp puts its pair into all CTAs of the
//                           cluster (a marked 64-bit word, no barrier), takes the next row's first
//                           chunks meanwhile, and combines all pairs in one order.  Pass B: the dense
//                           term g T q from the slots, which are handed back one by one.
// Measured at 2048 rows of 151936 bf16 logits (two CTAs per row, 152 KB each in a ring of 11 slots of
// 20 KB, one CTA per SM): 206 us for 1.24 GB, 6.0 TB/s, against 278 us for a statistics and a dense
// pass and 277 for one block per row that reads it twice, the second time from L2.  The consumers'
// instructions bound it (about nine per logit and lane, and each row's own work per warp): 16 warps
// 213 us, 24 219, four CTAs per row 256.
//
// Every wait has a limit.  A warp whose wait gave up waits no more and hands no slot back, so the
// producer and those that need its pairs end at their own limits; it walks the rest of its rows with
// whatever the slots hold (leaving the loop instead costs the kernel a third of its speed: 290 us).  At
// the end its whole cluster waits for the copies in flight and leaves all of its rows NaN.
#include "rows.cuh"
#include "sm100.cuh"

namespace dh {
namespace {

constexpr int DR_WARPS = 20;
constexpr int DR_NT = DR_WARPS * 32;            // consumers
constexpr int DR_THREADS = DR_NT + 32;          // and the producer's warp
constexpr int DR_MAX_C = 8;
constexpr int DR_MAX_SLOTS = 32;
constexpr int DR_CHUNK = 2 * DR_NT;             // vectors per chunk: two per thread
constexpr long long DR_LIMIT = 4000000000ll;    // cycles (two seconds) after which a wait gives up

struct RingArgs {
  DistillArgs d;
  int lg;       // C = 2^lg
  int slots;    // ring slots
  int spare;    // of them not needed by a row
  bool loose;   // rows may have elements beside their 16-byte grid
  long long limit;  // cycles after which a wait gives up
  RingTest test;
};

__device__ __forceinline__ void st16(void* p, const uint4& v) {
  asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t remote_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(sm100::smem_u32(p)), "r"(rank));
  return r;
}
// The pairs that the warps exchange, in one 64-bit word each: the maximum's bits, and the sum's with
// its last bit (2^-24 of it) given to a mark that changes whenever the slot is used again.  A word is
// written and read whole, so it carries its own arrival: no fence has to wait for the gradient's
// stores in flight, which one at cluster scope does (an earlier build took 262 us so, 247 without).
__device__ __forceinline__ unsigned long long pair_word(float m, float s, uint32_t mark) {
  return (unsigned long long)__float_as_uint(m) << 32 | ((__float_as_uint(s) & ~1u) | mark);
}
__device__ __forceinline__ void put_word(uint32_t dst, unsigned long long w) {
  asm volatile("st.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(dst), "l"(w) : "memory");
}
__device__ __forceinline__ unsigned long long get_word(const unsigned long long* p) {
  unsigned long long w;
  asm volatile("ld.relaxed.cluster.shared::cta.b64 %0, [%1];" : "=l"(w) : "r"(sm100::smem_u32(p)) : "memory");
  return w;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A CTA's share of a row: vectors [lo, hi) of the row's 16-byte grid, which starts at element `pre`
// and ends before element `behind`.  The first CTA also has the elements beside the grid.
struct Slice {
  int pre, behind, lo, hi;
};
template <typename T>
__device__ __forceinline__ Slice slice_of(const T* z, int vocab, int part, int lg) {
  Slice s;
  s.pre = min(vocab, (int)(((16u - (unsigned)(reinterpret_cast<uintptr_t>(z) & 15u)) & 15u) / sizeof(T)));
  const unsigned nvec = (unsigned)(vocab - s.pre) / Elem<T>::PER16;
  s.behind = s.pre + (int)nvec * Elem<T>::PER16;
  s.lo = (int)(nvec * (unsigned)part >> lg);
  s.hi = (int)(nvec * (unsigned)(part + 1) >> lg);
  return s;
}

// What a CTA does when a wait of its cluster has given up: it waits for its copies in flight (of slot i
// the last one was of parity `phase`, or the other one for i < slot) and leaves NaN in its part of the
// cluster's rows and in their statistics, whatever was written there.
template <typename T>
__device__ __noinline__ void abandon(const RingArgs& a, uint64_t* full, int slot, uint32_t phase, int part) {
  const DistillArgs& d = a.d;
  if (threadIdx.x == 0 && d.status) atomicOr(d.status, 1 << DH_ERR_TIMEOUT);
  if ((int)threadIdx.x < a.slots) {
    const uint32_t parity = (int)threadIdx.x < slot ? phase ^ 1u : phase;
    const long long t0 = clock64();
    while (!sm100::mbar_try_wait(&full[threadIdx.x], parity) && clock64() - t0 <= DR_LIMIT) {
    }
  }
  __syncthreads();
  const T nan = Elem<T>::from_f(NAN);
  for (long long row = blockIdx.x >> a.lg; row < d.N; row += gridDim.x >> a.lg) {
    const Slice s = slice_of(static_cast<const T*>(d.logits) + row * d.ld, d.vocab, part, a.lg);
    T* const out = static_cast<T*>(d.grad) + row * d.gld;
    const int lo = part == 0 ? 0 : s.pre + s.lo * Elem<T>::PER16, hi = s.pre + s.hi * Elem<T>::PER16;
    for (int i = lo + (int)threadIdx.x; i < hi; i += DR_THREADS) out[i] = nan;
    if (part != 0) continue;
    for (int i = s.behind + (int)threadIdx.x; i < d.vocab; i += DR_THREADS) out[i] = nan;
    if (threadIdx.x == 0) d.stats_out[row] = make_float2(NAN, NAN);
  }
}

// TEST: the form that the self-test runs (RingTest).
template <typename T, bool TEST>
__global__ void __launch_bounds__(DR_THREADS, 1) k_distill_ring(RingArgs a) {
  const DistillArgs& d = a.d;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  uint4* const ring = reinterpret_cast<uint4*>(ring_smem);         // [slots][DR_CHUNK]
  __shared__ __align__(16) unsigned long long s_pair[2][DR_MAX_C * DR_WARPS];  // every warp's pair
  __shared__ uint64_t full[DR_MAX_SLOTS], empty[DR_MAX_SLOTS];
  __shared__ uint32_t s_stop;         // a wait of the cluster has given up
  __shared__ uint32_t s_last[2];      // the producer's next slot and phase, once it is done

  const int lg = a.lg, C = 1 << lg, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cl = blockIdx.x >> lg, part = blockIdx.x & (C - 1), ncl = gridDim.x >> lg;
  const T* const logits = static_cast<const T*>(d.logits);

  if (tid == 0) {
    s_stop = 0;
    for (int i = 0; i < a.slots; ++i) {
      sm100::mbar_init(&full[i], 1);
      sm100::mbar_init(&empty[i], DR_WARPS);
    }
    sm100::fence_barrier_init();
  }
  for (int i = tid; i < 2 * DR_MAX_C * DR_WARPS; i += DR_THREADS) (&s_pair[0][0])[i] = 1ull;  // marked as not yet put
  __syncthreads();
  if (C > 1) cluster_barrier();  // the others' slots are there before anything is put
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // only now: the kernel after this one reads the call's inputs as soon as it may start
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  bool failed = false;
  // In a wait that started at t0: whether it is to end without what it waits for.
  auto give_up = [&](long long t0) {
    if (!failed && clock64() - t0 <= a.limit) return false;
    failed = true;
    *(volatile uint32_t*)&s_stop = 1;
    return true;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (failed || sm100::mbar_try_wait(bar, parity)) return;
    const long long t0 = clock64();
    while (!sm100::mbar_try_wait(bar, parity))
      if (give_up(t0)) return;
  };
  // What the self-test holds back, from a row on, in the cluster's last CTA
  auto held = [&](int what, long long row) {
    return TEST && a.test.hold == what && part == C - 1 && row >= a.test.row;
  };

  if (warp == DR_WARPS) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 1;  // the first round finds the slots free
      for (long long row = cl; row < d.N && !failed; row += ncl) {
        if (held(RingTest::COPIES, row)) break;
        const T* z = logits + row * d.ld;
        const Slice s = slice_of(z, d.vocab, part, lg);
        const uint4* src = reinterpret_cast<const uint4*>(z + s.pre) + s.lo;
        for (int v = 0; v < s.hi - s.lo; v += DR_CHUNK) {
          const uint32_t bytes = (uint32_t)min(DR_CHUNK, s.hi - s.lo - v) * 16u;
          wait(&empty[slot], phase);
          if (failed) break;
          sm100::mbar_arrive_expect_tx(&full[slot], bytes);
          sm100::bulk_load(ring + slot * DR_CHUNK, src + v, bytes, &full[slot]);
          if (++slot == a.slots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      s_last[0] = (uint32_t)slot;
      s_last[1] = phase;
    }
  } else {
    // ---------------------------------------------------------------- consumers
    int slot_a = 0, slot_b = 0, it = 0;
    uint32_t ph_a = 0;
    constexpr uint32_t NEG = NegInf<T>::WORD;
    // the element beside the grid that this thread holds, or -1
    auto beside = [&](const Slice& s) {
      if (!a.loose || part != 0 || warp != 0) return -1;
      const int at = tid < s.pre ? tid : s.behind + tid - s.pre;
      return at < d.vocab ? at : -1;
    };
    // A row's pass A as far as it has come: running maximum and sum, vectors done, and the element
    // beside the grid.
    struct RowState {
      float m, s, x;
      int v;
    };
    auto begin = [&](long long row) {
      RowState r = {-INFINITY, 0.f, -INFINITY, 0};
      if (row < d.N && a.loose) {
        const T* z = logits + row * d.ld;
        const int at = beside(slice_of(z, d.vocab, part, lg));
        if (at >= 0) r.m = r.x = Elem<T>::to_f(*(const volatile T*)(z + at));
        if (r.x != -INFINITY) r.s = row_ex2((r.x - r.x) * d.c);  // 1, or NaN
      }
      return r;
    };
    RowState next = begin(cl);
    for (long long row = cl; row < d.N; row += ncl, ++it) {
      const int par = it & 1;
      const Slice sl = slice_of(logits + row * d.ld, d.vocab, part, lg);
      const int nl = sl.hi - sl.lo, lone = beside(sl);
      const float g = __ldg(d.weight + row) * d.temperature;
      const bool zero = g == 0.f || (d.n_valid && __ldg(d.n_valid + row) <= 0);
      float m = next.m, s = next.s;
      const float x = next.x;
      // two chunks at a time, four independent vectors per thread; whole ones without bounds checks
      auto take = [&](const uint4 (&u)[4], float& m, float& s) {
        const float mn = max_nan(m, vec_max<T>(u));
        if (mn != m) {
          s = m == -INFINITY ? 0.f : s * row_ex2((m - mn) * d.c);
          m = mn;
        }
        if (m != -INFINITY) {
          const ExpRef ref(m, d.c);
          float t[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = vec_expsum<T>(u[i], ref, d.c);
          s += ref.by_max((t[0] + t[1]) + (t[2] + t[3]), d.c);
        }
      };
      auto next_a = [&] {
        if (++slot_a == a.slots) {
          slot_a = 0;
          ph_a ^= 1;
        }
      };
      auto take_two = [&](float& m, float& s) {
        uint4 u[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4* const b = ring + slot_a * DR_CHUNK + tid;
          wait(&full[slot_a], ph_a);
          u[2 * h] = b[0];
          u[2 * h + 1] = b[DR_NT];
          next_a();
        }
        take(u, m, s);
      };
      int v = next.v;
      for (; v + 2 * DR_CHUNK <= nl; v += 2 * DR_CHUNK) take_two(m, s);
      if (v < nl) {
        uint4 u[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = nl - v - h * DR_CHUNK;  // may be negative: no chunk
          const uint4* const b = ring + slot_a * DR_CHUNK + tid;
          if (n > 0) wait(&full[slot_a], ph_a);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            u[2 * h + i] = tid + i * DR_NT < n ? b[i * DR_NT] : make_uint4(NEG, NEG, NEG, NEG);
          if (n > 0) next_a();
        }
        take(u, m, s);
      }
      // the warp's pair, then everybody's
      const float wm = warp_max(m);
      s = m == -INFINITY ? 0.f : s * row_ex2((m - wm) * d.c);
      s = warp_sum(s);
      const uint32_t mark = (it >> 1) & 1;
      if (lane < C && !(held(RingTest::PAIRS, row) && warp == 0)) {
        const unsigned long long word = pair_word(wm, s, mark);
        if (C == 1) *reinterpret_cast<volatile unsigned long long*>(&s_pair[par][warp]) = word;
        else put_word(remote_addr(&s_pair[par][part * DR_WARPS + warp], lane), word);
      }
      // while the pairs travel: the next row's first chunks, as far as the ring holds them beside this
      // row's (a.spare) and they are there
      next = begin(row + ncl);
      if (a.spare >= 2 && row + ncl < d.N) {
        const Slice ns = slice_of(logits + (row + ncl) * d.ld, d.vocab, part, lg);
        const int most = min(ns.hi - ns.lo, a.spare * DR_CHUNK) - 2 * DR_CHUNK;
        while (next.v <= most) {
          const int second = slot_a + 1 == a.slots ? 0 : slot_a + 1;
          const bool there = sm100::mbar_try_wait(&full[slot_a], ph_a) &&
                             sm100::mbar_try_wait(&full[second], second ? ph_a : ph_a ^ 1);
          if (!__all_sync(0xFFFFFFFFu, there)) break;
          take_two(next.m, next.s);
          next.v += 2 * DR_CHUNK;
        }
      }
      const long long t0 = clock64();
      m = -INFINITY;
      s = 0.f;
      for (int i = lane; i < C * DR_WARPS; i += 32) {  // lane by lane in a fixed order
        unsigned long long word = get_word(&s_pair[par][i]);
        while (((uint32_t)word & 1u) != mark && !give_up(t0)) word = get_word(&s_pair[par][i]);
        const float pm = __uint_as_float((uint32_t)(word >> 32)), ps = __uint_as_float((uint32_t)word & ~1u);
        const float mn = max_nan(m, pm);
        s = (m == -INFINITY ? 0.f : s * row_ex2((m - mn) * d.c)) +
            (pm == -INFINITY ? 0.f : ps * row_ex2((pm - mn) * d.c));
        m = mn;
      }
      __syncwarp();
      failed = __any_sync(0xFFFFFFFFu, failed);
      const float lm = m;
      m = warp_max(m);
      s = warp_sum(lm == -INFINITY ? 0.f : s * row_ex2((lm - m) * d.c));
      if (part == 0 && tid == 0) d.stats_out[row] = make_float2(m, s);

      T* const out = static_cast<T*>(d.grad) + row * d.gld;
      const bool nothing = m == -INFINITY;  // a row of -inf has q = 0
      const ExpRef ref(nothing ? 0.f : m, d.c);
      const float aq = nothing ? 0.f : ref.by_max(g / s, d.c);
      uint4* o = reinterpret_cast<uint4*>(out + sl.pre) + sl.lo + tid;
      auto next_b = [&] {  // the slot is read: it goes back to the producer
        if (lane == 0 && !failed && !(held(RingTest::SLOTS, row) && warp == 0)) sm100::mbar_arrive(&empty[slot_b]);
        if (++slot_b == a.slots) slot_b = 0;
      };
      v = 0;
      for (; v + 2 * DR_CHUNK <= nl && !zero; v += 2 * DR_CHUNK, o += 2 * DR_CHUNK) {
        uint4 u[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4* const b = ring + slot_b * DR_CHUNK + tid;
          u[2 * h] = b[0];
          u[2 * h + 1] = b[DR_NT];
          __syncwarp();
          next_b();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) st16(o + i * DR_NT, grad_vec<T>(u[i], ref, d.c, aq));
      }
      for (; v < nl; v += DR_CHUNK, o += DR_CHUNK) {
        const int n = nl - v;
        uint4 u[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (tid + i * DR_NT < n) u[i] = ring[slot_b * DR_CHUNK + tid + i * DR_NT];
        __syncwarp();
        next_b();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (tid + i * DR_NT < n)
            st16(o + i * DR_NT, zero ? make_uint4(0, 0, 0, 0) : grad_vec<T>(u[i], ref, d.c, aq));
      }
      if (lone >= 0) out[lone] = Elem<T>::from_f(zero ? 0.f : aq * one_exp(x, ref, d.c));
    }
  }
  __syncthreads();
  if (C > 1) {
    if (*(const volatile uint32_t*)&s_stop != 0 && tid < C)
      asm volatile("st.relaxed.cluster.shared::cluster.b32 [%0], %1;" ::"r"(remote_addr(&s_stop, tid)), "r"(1)
                   : "memory");
    cluster_barrier();  // no CTA leaves while another may still put something into it
  }
  if (*(const volatile uint32_t*)&s_stop != 0) abandon<T>(a, full, (int)s_last[0], s_last[1], part);
}

template <typename T, bool TEST>
cudaError_t run(const Ctx& c, const DistillArgs& d, const RingTest* test, bool* done) {
  *done = false;
  auto* kernel = k_distill_ring<T, TEST>;
  static unsigned long long smem_done = 0;
  cudaError_t e = allow_max_smem(kernel, c.device, &smem_done);
  if (e == cudaSuccess) e = carveout_max_shared((const void*)kernel, c.device);
  if (e != cudaSuccess) return e;
  static int dyn_max[64] = {};
  const int dv = c.device < 64 ? c.device : 0;
  if (dyn_max[dv] == 0 || c.device >= 64) dyn_max[dv] = max_dynamic_smem(kernel, c.device);

  RingArgs a = {};
  a.d = d;
  a.limit = DR_LIMIT;
  if (TEST) {
    a.test = *test;
    a.limit = 2000ll * test->limit_us;  // about 2 GHz
  }
  const int vecs = d.vocab / Elem<T>::PER16;
  // The cut: the fewest CTAs that hold a row with a slot to spare, then more while the rows alone do
  // not fill the SMs.
  bool fits = false;
  for (a.lg = 0; a.lg <= 3; ++a.lg) {
    const int slice = (vecs >> a.lg) > 0 ? (vecs + (1 << a.lg) - 1) >> a.lg : 1;
    const int chunks = (slice + DR_CHUNK - 1) / DR_CHUNK;
    const int slots = dyn_max[dv] / (16 * DR_CHUNK);
    a.slots = slots < DR_MAX_SLOTS ? slots : DR_MAX_SLOTS;
    a.spare = a.slots - chunks;
    fits = a.spare >= 1;
    if (fits && ((long long)d.N << a.lg >= c.num_sms || slice <= 512 || a.lg == 3)) break;
  }
  if (!fits) return cudaSuccess;
  const int C = 1 << a.lg;
  a.loose = !rows_aligned(d.logits, d.ld, 0, d.N, 1, (int)sizeof(T)) || d.vocab % Elem<T>::PER16 != 0;
  *done = true;

  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C);
  cfg.blockDim = dim3(DR_THREADS);
  cfg.dynamicSmemBytes = (size_t)a.slots * DR_CHUNK * 16;
  cfg.stream = c.stream;
  cfg.attrs = at;
  int fit = c.num_sms / C;
  if (C > 1) {
    static int clusters[64][4] = {};  // that run at once
    if (clusters[dv][a.lg] == 0 || c.device >= 64) {
      cudaLaunchConfig_t q = cfg;
      q.attrs = at + 1;
      q.numAttrs = 1;
      q.dynamicSmemBytes = dyn_max[dv];
      e = cudaOccupancyMaxActiveClusters(&clusters[dv][a.lg], kernel, &q);
      if (e != cudaSuccess) return e;
    }
    fit = clusters[dv][a.lg];
  }
  if (fit < 1) fit = 1;
  cfg.gridDim = dim3((unsigned)((d.N < fit ? d.N : fit) * C));
  cfg.numAttrs = C > 1 ? 2 : 1;
  prof_before("distill_ring", c.stream);
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  prof_after(c.stream);
  return e;
}

}  // namespace

cudaError_t launch_distill_ring(const Ctx& c, const DistillArgs& a, int dtype, bool* done, const RingTest* test) {
  if (test) return dtype == DH_F32 ? run<float, true>(c, a, test, done) : cudaErrorInvalidValue;
  return dtype == DH_BF16 ? run<__nv_bfloat16, false>(c, a, nullptr, done) : run<float, false>(c, a, nullptr, done);
}

}  // namespace dh
