// Decode attention of one new token per request over a paged key-value cache.
//
// Per request m and q head h of kv head g, over the positions j it attends to (its length, or the
// window at its end):
//   s_j = scale q . k_j,   o = sum_j exp(s_j - ref) v_j / sum_j exp(s_j - ref),   lse = ref + ln sum
// in one pass with a running reference instead of a second look: ref is the maximum of the first
// chunk, and where a later score is above it by more than a step (kStep, in powers of two) the new
// maximum takes its place and what was summed is scaled down.  Scores are held times log2 e, for ex2.
//
// HBM-bound: the cache is read once, 4 flops per q head and element.  One persistent CTA per SM; the
// work is a list of units (request, kv head, chunk of 128 positions) split evenly over the CTAs in
// order, so that one long request and many short ones load all SMs alike.  Both products run on
// tcgen05 with the cache as the 128-row operand, straight from where TMA put it:
//   S^T [128 positions, 16 heads] = K Q^T      K as it lies (rows of positions), Q padded to 16 heads
//   O^T [dims, 16 heads]         += V^T P^T    V as it lies too, read as the transposed operand
// so no byte of k or v passes through registers.  A thread of the softmax warps holds one position
// and half of the heads; maxima are looked for across threads only when a score passes the step.
//   bf16 pages: P enters the product as two bf16 (its rounding and the rest), so that P's rounding
//     does not show beside the output's own; the tensor cores have the time.
//   e4m3 pages: e4m3 products (kind::f8f6f4).  q is split into two codes (q / 2^e = hi + lo, all of a
//     bf16's bits unless it is below 2^-10 of its head's largest value).  P is split into three, each the
//     rest of the one before times 16: good to 2^-12 of its value or 2^-25 of a weight of 1, so that
//     the many small weights of a long context are not lost.  The heads' scales go to the scores and to
//     the output.
// The codes of a split operand are columns of one MMA side by side (N = 16 per code) and their products
// are added when tensor memory is read: an MMA costs the 128-row operand's way out of shared memory,
// whatever N is, so a code more costs nothing and an MMA more does (62 cycles alone, 150 beside TMA's
// writes; one MMA per code took 120.8 us for 131071 tokens of the 70B heads).
// Warps: 0-7 softmax, 8 TMA producer (lane i looks up the page of box i and copies it: 16 to 128
// positions by 128 bytes), 9 issues the scores' MMAs and 11 those of P V, each as soon as its operands are
// there (one thread for both made every chunk wait for the one before: 107.1 us instead of 95.5 for 131071 tokens),
// 10 brings the q of the next (request, kv head).
// A (request, kv head) that is split over CTAs leaves a piece per CTA (sum of p v, ref, sum) and the
// CTA that counts in last joins the pieces in order.  Every sum's order follows from the lengths and
// the SM count: runs repeat bit for bit.
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "attn_mma.cuh"
#include "common.cuh"
#include "paged.h"
#include "tc.h"
#include "tc_ptx.cuh"

namespace tpx {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kP = 128;                    // positions per chunk: the rows of an MMA
constexpr int kN = 16;                     // heads of an MMA (its columns)
constexpr int kSoft = 256;                 // softmax threads
constexpr int kThreads = kSoft + 128;      // and the producer, the q warp and one MMA warp per product
constexpr int kMasks = 32;                 // ring of the chunks' masks: above the chunks in flight

template <int HD, bool FP8>
struct PCfg {
  static constexpr int ROWB = HD * (FP8 ? 1 : 2);                 // bytes of a position
  static constexpr int INB = ROWB < 128 ? ROWB : 128;             // bytes of a box row
  static constexpr int NIB = ROWB / INB;                          // boxes side by side
  static constexpr int STAGE = kP * ROWB;                         // k or v of a chunk
  static constexpr int NS = std::min(16, (192 * 1024) / STAGE);   // stages, k and v in turn
  static constexpr int NB = HD == 256 ? 2 : 1;                    // 128-dim blocks of O^T
  static constexpr int KS = FP8 ? 32 : 16;                        // k of an MMA
  static constexpr int TERMS = FP8 ? 3 : 2;                       // codes that P is split into
  static constexpr int PROW = kN * (FP8 ? 1 : 2);                 // bytes of a position of P
  static constexpr int PTILE = kP * PROW;
  static constexpr int QTERMS = FP8 ? 2 : 1;                      // codes of q, 16 rows each
  static constexpr int QBOX = QTERMS * kN * 128;                  // their rows' 128 bytes
  static constexpr int QTILE = (ROWB + 127) / 128 * QBOX;
  static constexpr float kStep = FP8 ? 1.f : 8.f;                 // ref may be behind the maximum by this
  static constexpr float kPMul = FP8 ? 128.f : 1.f;               // P is held times this: up to 256 in e4m3
  static constexpr float kNext = FP8 ? 16.f : 1.f;                // each code of P after the first is held times this
  static constexpr uint32_t kCols = FP8 || NB == 2 ? 256 : 128;   // TMEM: S [2][QTERMS][16], O [2][NB][TERMS][16]
  static_assert(2 * kN * (QTERMS + NB * TERMS) <= (int)kCols, "TMEM");
  static constexpr size_t kRing = (size_t)NS * STAGE;
  static constexpr size_t SMEM = 1024 + kRing + 2 * TERMS * PTILE + 2 * QTILE;
  static_assert(NS >= 3, "a chunk's k and v and the next one's k");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// what a sum taken under reference m counts under the reference mx (0 where nothing was summed)
__device__ __forceinline__ float weight(float m, float mx) { return m == -INFINITY ? 0.f : ex2(m - mx); }

// 32 lanes x N consecutive 32-bit columns of tensor memory; the values are there after landed()
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t t, float (&v)[N]) {
  uint32_t r[N];
  if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(t));
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
// Waits for the loads; the values pass through it, so that no use of them can move before.
template <int N>
__device__ __forceinline__ void landed(float (&v)[N]) {
  tc::tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t t, const float (&v)[N]) {
  if constexpr (N == 4) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t), "r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3]))
                 : "memory");
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
  }
  tc::tmem_st_wait();
}

// Shared-memory operand descriptor: strides in bytes, layout 2 / 4 / 6 / 0 = 128 / 64 / 32-byte swizzle / none.
// K-major: `stride` between 8-row groups.  Transposed (rows of k): `stride` between groups of 8 k,
// `lead` between the blocks of a swizzle row's length along the other side.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride, uint32_t layout) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((lead >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((stride >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)layout << 61;
}
constexpr uint32_t kTransposed = (1u << 15) | (1u << 16);  // instruction descriptor: A and B are rows of k

// named barriers of n threads; any(): whether the predicate holds for one of them
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool bar_any(int id, int n, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// two floats as e4m3 codes (x in the low byte), and back
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
  return __half22float2(__half2(h));
}

// The positions [lo, n) a request attends to, in chunks [c0, c1); c0 == c1 if there are none.
struct Span {
  int lo, n, c0, c1;
};
__device__ __forceinline__ Span span_of(const PagedAttnArgs& a, int m) {
  Span s{0, a.lens[m], 0, 0};
  if (s.n < 1 || (long long)s.n > ((long long)a.max_pages << a.page_shift)) return s;
  if (a.window > 0) s.lo = max(0, s.n - a.window);
  s.c0 = s.lo / kP;
  s.c1 = (s.n - 1) / kP + 1;
  return s;
}

// A unit: chunk c of (m, gg).  `seg` counts the (m, gg) that the CTA has begun.
struct Cursor {
  int m, gg, c, seg;
  Span s;
  __device__ __forceinline__ bool ends() const { return c + 1 == s.c1; }
};
__device__ __forceinline__ void advance(const PagedAttnArgs& a, Cursor& cu) {  // only when there is a next unit
  if (++cu.c < cu.s.c1) return;
  ++cu.seg;
  if (++cu.gg == a.n_kv) {
    cu.gg = 0;
    do {
      ++cu.m;
      cu.s = span_of(a, cu.m);
    } while (cu.s.c0 == cu.s.c1 && cu.m + 1 < a.M);
  }
  cu.c = cu.s.c0;
}
// Bits of the chunk's 16-position groups with a position that counts: within [lo, n) and loaded.
__device__ __forceinline__ uint32_t group_bits(const Cursor& cu, uint32_t loaded) {
  const int a0 = max(0, cu.s.lo - cu.c * kP), a1 = min(kP, cu.s.n - cu.c * kP);
  return loaded & ((1u << ((a1 + 15) >> 4)) - 1) & ~((1u << (a0 >> 4)) - 1);
}

// CTA i of nct (at most U) takes units [U i / nct, U (i + 1) / nct); owner(u) is the CTA of unit u.
__device__ __forceinline__ long long split_at(long long U, int nct, int i) { return U * i / nct; }
__device__ __forceinline__ int owner(long long U, int nct, long long u) {
  return (int)(((u + 1) * nct + U - 1) / U) - 1;
}

// A role's bounded waits: one that runs out sets the error word, and the role goes on without
// waiting, so that every barrier is still met and the kernel ends.
struct Waits {
  unsigned* err;
  unsigned code;
  bool failed;
  __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) {
    if (!failed && !tc::mbar_wait(bar, parity)) {
      atomicExch(err, code);
      failed = true;
    }
  }
};

// grid: one CTA per SM.  HPT: heads per softmax thread, 2 HPT >= n_q / n_kv.
template <int HD, bool FP8, int HPT>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ PagedAttnArgs a) {
  using C = PCfg<HD, FP8>;
  extern __shared__ __align__(1024) uint8_t sm_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = ring + C::kRing;                     // [2][QTILE]
  uint8_t* sP = sQ + 2 * C::QTILE;                  // [2][TERMS][PTILE]
  __shared__ __align__(8) uint64_t kv_full[2][C::NS], kv_empty[2][C::NS], q_full[2], q_empty[2], s_full[2], s_empty[2],
      p_full[2], p_empty[2], o_full[2], o_empty[2];
  __shared__ long long s_part[kThreads / 32], s_off;
  __shared__ float s_max[8][HPT], s_sum[8][HPT], q_pow[4][kN];
  __shared__ uint32_t loaded[kMasks];                // 16-position groups of a chunk that were loaded, by bit
  __shared__ uint32_t s_tmem;
  __shared__ int s_m, s_last[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  auto B = [](const uint64_t& b) { return tc::smem_u32(&b); };
  if (tid == 0) {
    for (int i = 0; i < 2 * C::NS; ++i) {
      tc::mbar_init(B(kv_full[i & 1][i >> 1]), 1);
      tc::mbar_init(B(kv_empty[i & 1][i >> 1]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(B(q_full[i]), 1);
      tc::mbar_init(B(q_empty[i]), 1);
      tc::mbar_init(B(s_full[i]), 2);  // the MMAs' commit, and the issuing thread's own arrival
      tc::mbar_init(B(s_empty[i]), kSoft / 32);
      tc::mbar_init(B(p_full[i]), kSoft / 32);
      tc::mbar_init(B(p_empty[i]), 1);
      tc::mbar_init(B(o_full[i]), 1);
      tc::mbar_init(B(o_empty[i]), kSoft / 32);
    }
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  for (int i = tid; i < 2 * C::TERMS * C::PTILE / 16; i += kThreads)  // P of heads that no thread holds stays 0
    reinterpret_cast<uint4*>(sP)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  const int G = a.n_q / a.n_kv, nkvs = a.n_kv / a.t;

  // rows without positions
  for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
    const Span s = span_of(a, m);
    if (s.c0 != s.c1) continue;
    uint4* o = reinterpret_cast<uint4*>(a.o + (size_t)m * a.n_q * HD);
    for (int i = tid; i < a.n_q * HD / 8; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = tid; i < a.n_q; i += kThreads) a.lse[(size_t)m * a.n_q + i] = -INFINITY;
  }

  // the units: a sum over the requests, a contiguous run of them per thread
  const int per = (a.M + kThreads - 1) / kThreads, r0 = min(a.M, tid * per), r1 = min(a.M, r0 + per);
  long long here = 0;
  for (int m = r0; m < r1; ++m) {
    const Span s = span_of(a, m);
    here += s.c1 - s.c0;
  }
  long long incl = here;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) s_part[warp] = incl;
  __syncthreads();
  long long U = 0, before = incl - here;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s_part[w];
    U += s_part[w];
  }
  U *= a.n_kv;
  const int nct = (int)min((long long)gridDim.x, U);
  if ((int)blockIdx.x >= nct) return;
  const long long u0 = split_at(U, nct, blockIdx.x), u1 = split_at(U, nct, blockIdx.x + 1);
  if (u0 >= before * a.n_kv && u0 < (before + here) * a.n_kv) {  // this thread's requests hold unit u0
    int m = r0;
    long long off = u0 - before * a.n_kv;
    for (;; ++m) {
      const Span s = span_of(a, m);
      const long long n = (long long)(s.c1 - s.c0) * a.n_kv;
      if (off < n) break;
      off -= n;
    }
    s_m = m;
    s_off = off;
  }
  if (warp == 9) tc::tmem_alloc(tc::smem_u32(&s_tmem), C::kCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto S_at = [&](int k, int term) { return tmem + ((k & 1) * C::QTERMS + term) * kN; };
  auto O_at = [&](int seg, int nb, int term) {
    return tmem + (2 * C::QTERMS + ((seg & 1) * C::NB + nb) * C::TERMS + term) * kN;
  };
  const int nu = (int)(u1 - u0);
  Cursor cu;
  cu.m = s_m;
  cu.seg = 0;
  cu.s = span_of(a, cu.m);
  cu.gg = (int)(s_off / (cu.s.c1 - cu.s.c0));
  cu.c = cu.s.c0 + (int)(s_off % (cu.s.c1 - cu.s.c0));

  // pieces of a split (request, kv head): only this CTA's first or last can be one
  int np_mine = 0, pm[2], pgg[2], pa[2], pb[2];
  bool pst[2];  // the first of its CTAs starts with it
  float* part = reinterpret_cast<float*>(a.ws + kPagedMaxCtas);
  const int per_piece = (G * (HD + 2) + 3) / 4 * 4;

  constexpr uint32_t kLay = C::INB == 128 ? 2 : 4;  // swizzle of the cache's stages
  auto mma = [](uint32_t d, uint64_t x, uint64_t y, uint32_t id, bool acc) {
    if (FP8) tc::mma_e4m3(d, x, y, id, acc);
    else tc::mma_bf16(d, x, y, id, acc);
  };

  if (warp == 8) {
    // ---- producer: k of chunk c in stage 2 c, v in 2 c + 1 (modulo NS).  The barriers go by (k or v, chunk
    // modulo NS), not by stage: each is then waited for phase by phase by one role (with an odd NS a
    // stage holds k and v in turn, and the role that reads k would miss every other phase).
    Waits wait{a.err, 44u, false};
    const int box_rows = min(1 << a.page_shift, kP), nbp = kP / box_rows;  // boxes along the positions
    const int box = lane % nbp, side = lane / nbp;
    const uint64_t pol = tc::l2_evict_first();  // the cache streams through once
    auto page_of = [&](const Cursor& x) {  // the page id of this lane's box, -1: nothing to load
      const int p = x.c * kP + box * box_rows;
      if (side >= C::NIB || p >= x.s.n || p + box_rows <= x.s.lo) return -1;
      return a.table[(size_t)x.m * a.table_stride + (p >> a.page_shift)];
    };
    int id = page_of(cu);
    for (int k = 0; k < nu; ++k) {
      Cursor nx = cu;
      if (k + 1 < nu) advance(a, nx);
      const int next_id = k + 1 < nu ? page_of(nx) : -1;  // in flight while the stages are waited for
      const bool load = id >= 0 && id < a.n_pages;
      const unsigned boxes = __ballot_sync(kFull, load);
      const unsigned groups = __ballot_sync(kFull, lane < 8 && (boxes >> ((lane & 7) * 16 / box_rows) & 1));
      const int p = cu.c * kP + box * box_rows;
      const int row = ((((cu.gg / nkvs) * a.n_pages + id) * nkvs + cu.gg % nkvs) << a.page_shift) +
                      (p & ((1 << a.page_shift) - 1));
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int i = 2 * k + kv, st = i % C::NS;
        const int was = (i - C::NS) >> 1;  // the chunk whose k or v was in this stage
        if (i >= C::NS) wait(B(kv_empty[(i - C::NS) & 1][was % C::NS]), (was / C::NS) & 1);
        __syncwarp();
        if (lane == 0) {
          if (kv == 0) loaded[k % kMasks] = groups;
          tc::mbar_arrive_expect_tx(B(kv_full[kv][k % C::NS]), __popc(boxes) * box_rows * C::INB);
        }
        __syncwarp();
        if (load)
          tc::tma_load_2d_hint(tc::smem_u32(ring + (size_t)st * C::STAGE) + (side * kP + box * box_rows) * C::INB,
                               kv ? &tmV : &tmK, side * (C::INB / (FP8 ? 1 : 2)), row, B(kv_full[kv][k % C::NS]), pol);
      }
      cu = nx;
      id = next_id;
    }
  } else if (warp == 9) {
    // ---- scores: one thread issues
    if (lane == 0) {
      Waits wait{a.err, 45u, false};
      const uint32_t idesc = FP8 ? tc::idesc_e4m3(128, kN * C::QTERMS) : tc::idesc_bf16(128, kN * C::QTERMS);
      for (int k = 0; k < nu; ++k) {
        const int st = 2 * k % C::NS, qb = cu.seg & 1;
        wait(B(q_full[qb]), (cu.seg >> 1) & 1);
        wait(B(kv_full[0][k % C::NS]), (k / C::NS) & 1);
        if (k >= 2) wait(B(s_empty[k & 1]), ((k >> 1) - 1) & 1);
        tc::tc_fence_after();
        const uint32_t kA = tc::smem_u32(ring + (size_t)st * C::STAGE);
        const uint32_t qA = tc::smem_u32(sQ + (size_t)qb * C::QTILE);
#pragma unroll
        for (int i = 0; i < C::ROWB / 32; ++i) {  // 32 bytes of a row per MMA
          const uint32_t ka = kA + (32 * i) / C::INB * (kP * C::INB) + (32 * i) % C::INB;
          const uint32_t qa = qA + i / 4 * C::QBOX + (i % 4) * 32;
          mma(S_at(k, 0), smem_desc(ka, 16, 8 * C::INB, kLay), smem_desc(qa, 16, 1024, 2), idesc, i > 0);
        }
        tc::mma_commit(B(kv_empty[0][k % C::NS]));
        tc::mma_commit(B(s_full[k & 1]));
        tc::mbar_arrive(B(s_full[k & 1]));  // releases what this thread has seen: the chunk's mask
        if (k + 1 == nu || cu.ends()) tc::mma_commit(B(q_empty[qb]));
        if (k + 1 < nu) advance(a, cu);
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // ---- P V: one thread issues
    if (lane == 0) {
      Waits wait{a.err, 48u, false};
      const uint32_t idesc =
          (FP8 ? tc::idesc_e4m3(128, kN * C::TERMS) : tc::idesc_bf16(128, kN * C::TERMS)) | kTransposed;
      bool live = false;  // O of the (request, kv head) holds something
      for (int k = 0; k < nu; ++k) {
        const int st = (2 * k + 1) % C::NS, ob = cu.seg & 1;
        if (k == 0 || cu.c == cu.s.c0) {
          if (cu.seg >= 2) wait(B(o_empty[ob]), ((cu.seg >> 1) - 1) & 1);
          live = false;
        }
        wait(B(p_full[k & 1]), (k >> 1) & 1);
        wait(B(kv_full[1][k % C::NS]), (k / C::NS) & 1);
        tc::tc_fence_after();
        const uint32_t groups = group_bits(cu, loaded[k % kMasks]);
        const uint32_t vA = tc::smem_u32(ring + (size_t)st * C::STAGE);
        const uint32_t pA = tc::smem_u32(sP + (size_t)(k & 1) * C::TERMS * C::PTILE);
#pragma unroll
        for (int i = 0; i < kP / C::KS; ++i) {
          if (!(groups >> (i * C::KS / 16) & (FP8 ? 3u : 1u))) continue;
          // P's codes are tiles one after another: the blocks of its columns
          const uint32_t pt = pA + i * C::KS * C::PROW;
          const uint64_t pd = FP8 ? smem_desc(pt, 128, C::PTILE, 0) : smem_desc(pt, C::PTILE, 256, 6);
#pragma unroll
          for (int nb = 0; nb < C::NB; ++nb) {
            // a head of 64 dims fills half of the 128 rows: the other half reads it again (lead 0)
            const uint32_t va = vA + nb * (128 * (FP8 ? 1 : 2) / C::INB) * (kP * C::INB) + i * C::KS * C::INB;
            mma(O_at(cu.seg, nb, 0), smem_desc(va, HD == 64 ? 0 : kP * C::INB, 8 * C::INB, kLay), pd, idesc, live);
          }
          live = true;
        }
        tc::mma_commit(B(kv_empty[1][k % C::NS]));
        tc::mma_commit(B(p_empty[k & 1]));
        if (k + 1 == nu || cu.ends()) tc::mma_commit(B(o_full[ob]));
        if (k + 1 < nu) advance(a, cu);
      }
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---- q of each (request, kv head): G heads as 16 rows of 128-byte-swizzled pieces
    Waits wait{a.err, 46u, false};
    constexpr int RP = HD / 8;       // 16-byte pieces of a row: 8, 16 or 32 neighbouring lanes
    constexpr int QV = 16 * RP / 32;
    for (int k = 0; k < nu; ++k) {
      if (k == 0 || cu.c == cu.s.c0) {
        const __nv_bfloat16* qp = a.q + ((size_t)cu.m * a.n_q + (size_t)cu.gg * G) * HD;
        uint4 qn[QV];
#pragma unroll
        for (int i = 0; i < QV; ++i) {
          const int idx = lane + 32 * i, r = idx / RP, c8 = idx % RP;
          qn[i] = r < G ? *reinterpret_cast<const uint4*>(qp + (size_t)r * HD + 8 * c8) : make_uint4(0, 0, 0, 0);
        }
        const int qb = cu.seg & 1;
        if (cu.seg >= 2) wait(B(q_empty[qb]), ((cu.seg >> 1) - 1) & 1);
        uint8_t* dst = sQ + (size_t)qb * C::QTILE;
#pragma unroll
        for (int i = 0; i < QV; ++i) {
          const int idx = lane + 32 * i, r = idx / RP, c8 = idx % RP;
          if (FP8) {  // q / 2^e below 256, as two codes
            const uint32_t w[4] = {qn[i].x, qn[i].y, qn[i].z, qn[i].w};
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max((w[j] >> 7) & 0xffu, (w[j] >> 23) & 0xffu));
#pragma unroll
            for (int o = 1; o < RP; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
            // exponent field of the largest value, less 7 for 2^7 <= q / 2^e < 2^8; both factors stay normal
            const int e = min(max((int)top, 8), 253) - 7;
            const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
            uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float x = bf16_lo(w[j]) * inv, y = bf16_hi(w[j]) * inv;
              const uint32_t h = e4m3x2(x, y);
              const float2 b = e4m3x2_value(h);
              hi[j >> 1] |= h << (16 * (j & 1));
              lo[j >> 1] |= e4m3x2(x - b.x, y - b.y) << (16 * (j & 1));
            }
            uint8_t* at = dst + c8 / 16 * C::QBOX + r * 128 + (((c8 / 2 % 8) ^ (r & 7)) << 4) + (c8 & 1) * 8;
            *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(at + kN * 128) = make_uint2(lo[0], lo[1]);
            if (c8 == 0) q_pow[cu.seg & 3][r] = __uint_as_float((uint32_t)e << 23);
          } else {
            *reinterpret_cast<uint4*>(dst + c8 / 8 * C::QBOX + r * 128 + (((c8 % 8) ^ (r & 7)) << 4)) = qn[i];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(B(q_full[qb]));
      }
      if (k + 1 < nu) advance(a, cu);
    }
  } else {
    // ---- softmax: thread = position 32 (warp % 4) + lane and heads [h0, h0 + HPT); for O, dim and heads
    Waits wait{a.err, 47u, false};
    const int quad = warp & 3, half = warp >> 2, h0 = half * HPT, row = 32 * quad + lane, bid = 1 + half;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    float ref[HPT], l[HPT], sc[HPT];
    int c_seg = cu.c;      // first chunk of the current piece
    bool first_seg = true, fresh = true, live = false;  // fresh: at the piece's first chunk; live: O holds something
    for (int k = 0; k < nu; ++k) {
      wait(B(s_full[k & 1]), (k >> 1) & 1);
      tc::tc_fence_after();
      float s[HPT];
      tmem_ld<HPT>(S_at(k, 0) + h0 + lanes, s);
      if (C::QTERMS == 2) {
        float lo[HPT];
        tmem_ld<HPT>(S_at(k, 1) + h0 + lanes, lo);
        landed(lo);
        landed(s);
#pragma unroll
        for (int h = 0; h < HPT; ++h) s[h] += lo[h];
      } else {
        landed(s);
      }
      tc::tc_fence_before();
      if (fresh) {
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
          sc[h] = a.scale * kLog2e;
          if (FP8) sc[h] *= (a.k_scale ? a.k_scale[cu.gg] : 1.0f) * q_pow[cu.seg & 3][h0 + h];
          ref[h] = -INFINITY;
          l[h] = 0.f;
        }
        fresh = live = false;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(B(s_empty[k & 1]));
      const uint32_t groups = group_bits(cu, loaded[k % kMasks]);
      const int p = cu.c * kP + row;
      const bool counts = p >= cu.s.lo && p < cu.s.n && (groups >> (row >> 4) & 1);
      bool above = false;
#pragma unroll
      for (int h = 0; h < HPT; ++h) {
        s[h] = counts ? s[h] * sc[h] : -INFINITY;
        above |= s[h] > ref[h] + C::kStep;
      }
      if (bar_any(bid, kSoft / 2, above)) {  // a new reference: the maximum so far
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
          float x = s[h];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
          if (lane == 0) s_max[warp][h] = x;
        }
        bar_sync(bid, kSoft / 2);
        float f[HPT];
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
          float x = ref[h];
#pragma unroll
          for (int w = 0; w < 4; ++w) x = fmaxf(x, s_max[4 * half + w][h]);
          f[h] = weight(ref[h], x);
          l[h] *= f[h];
          ref[h] = x;
        }
        if (live) {  // once the P V before has ended
          wait(B(p_empty[(k - 1) & 1]), ((k - 1) >> 1) & 1);
          tc::tc_fence_after();
#pragma unroll
          for (int i = 0; i < C::NB * C::TERMS; ++i) {
            const uint32_t at = O_at(cu.seg, i / C::TERMS, i % C::TERMS) + h0 + lanes;
            float o[HPT];
            tmem_ld<HPT>(at, o);
            landed(o);
#pragma unroll
            for (int h = 0; h < HPT; ++h) o[h] *= f[h];
            tmem_st<HPT>(at, o);
          }
          tc::tc_fence_before();
        }
      }
#pragma unroll
      for (int h = 0; h < HPT; ++h) {  // a head without a score yet has reference -inf and weights 0
        s[h] = ex2(s[h] - (ref[h] == -INFINITY ? 0.f : ref[h]));
        l[h] += s[h];
      }
      if (k >= 2) wait(B(p_empty[k & 1]), ((k >> 1) - 1) & 1);
      uint8_t* pt = sP + (size_t)(k & 1) * C::TERMS * C::PTILE;
      if (FP8) {
        float r[HPT];
#pragma unroll
        for (int h = 0; h < HPT; ++h) r[h] = s[h] * C::kPMul;
#pragma unroll
        for (int t = 0; t < C::TERMS; ++t) {
          uint32_t w[HPT / 4];
#pragma unroll
          for (int i = 0; i < HPT / 4; ++i) {
            const uint32_t c0 = e4m3x2(r[4 * i], r[4 * i + 1]), c1 = e4m3x2(r[4 * i + 2], r[4 * i + 3]);
            w[i] = c0 | c1 << 16;
            if (t + 1 < C::TERMS) {
              const float2 x = e4m3x2_value(c0), y = e4m3x2_value(c1);
              r[4 * i] = (r[4 * i] - x.x) * C::kNext;
              r[4 * i + 1] = (r[4 * i + 1] - x.y) * C::kNext;
              r[4 * i + 2] = (r[4 * i + 2] - y.x) * C::kNext;
              r[4 * i + 3] = (r[4 * i + 3] - y.y) * C::kNext;
            }
          }
          uint8_t* at = pt + t * C::PTILE + row * 16 + h0;
          if constexpr (HPT == 8) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
          else *reinterpret_cast<uint32_t*>(at) = w[0];
        }
      } else {
        uint32_t hi[HPT / 2], lo[HPT / 2];
#pragma unroll
        for (int i = 0; i < HPT / 2; ++i) {
          const float x = s[2 * i], y = s[2 * i + 1];
          hi[i] = pack_bf16(x, y);
          lo[i] = pack_bf16(x - bf16_lo(hi[i]), y - bf16_hi(hi[i]));
        }
        // 32-byte rows, the two 16-byte pieces swapped in every other group of four rows
        uint8_t* at = pt + row * 32 + (((h0 >> 3) ^ ((row >> 2) & 1)) << 4) + (h0 & 7) * 2;
        if constexpr (HPT == 8) {
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(at + C::PTILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        } else {
          *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(at + C::PTILE) = make_uint2(lo[0], lo[1]);
        }
      }
      // v rows that do not count may hold anything (NaN too): where their MMA step runs, P V must see 0
      const bool step_runs = groups >> (row / C::KS * C::KS / 16) & (FP8 ? 3u : 1u);
      if (__any_sync(kFull, step_runs && !counts)) {
        const int st = (2 * k + 1) % C::NS;
        wait(B(kv_full[1][k % C::NS]), (k / C::NS) & 1);
        if (step_runs && !counts) {
          constexpr int PB = C::INB / 16, NPC = C::ROWB / 16;  // a row's pieces stay within it under any swizzle
          uint8_t* v = ring + (size_t)st * C::STAGE + row * C::INB;
#pragma unroll
          for (int j = 0; j < NPC / 2; ++j) {
            const int q = half * (NPC / 2) + j;
            *reinterpret_cast<uint4*>(v + q / PB * (kP * C::INB) + (q % PB) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
      }
      live |= groups != 0;
      fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(B(p_full[k & 1]));

      const bool last = k + 1 == nu, end = last || cu.ends();
      if (end) {  // the piece of (m, gg) in this CTA ends
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) l[h] += __shfl_xor_sync(kFull, l[h], o);
          if (lane == 0) s_sum[warp][h] = l[h];
        }
        bar_sync(bid, kSoft / 2);
#pragma unroll
        for (int h = 0; h < HPT; ++h)
          l[h] = (s_sum[4 * half][h] + s_sum[4 * half + 1][h]) + (s_sum[4 * half + 2][h] + s_sum[4 * half + 3][h]);
        const bool whole = c_seg == cu.s.c0 && cu.ends();
        const size_t orow = (size_t)cu.m * a.n_q + (size_t)cu.gg * G;  // of o and lse
        float* piece = part + (size_t)(2 * blockIdx.x + (first_seg ? 0 : 1)) * per_piece;
        const float vs = (FP8 && a.v_scale ? a.v_scale[cu.gg] : 1.0f) / C::kPMul;
        wait(B(o_full[cu.seg & 1]), (cu.seg >> 1) & 1);
        tc::tc_fence_after();
        float o[C::NB][HPT], ot[C::NB][C::TERMS][HPT];
#pragma unroll
        for (int i = 0; i < C::NB * C::TERMS; ++i)
          tmem_ld<HPT>(O_at(cu.seg, i / C::TERMS, i % C::TERMS) + h0 + lanes, ot[i / C::TERMS][i % C::TERMS]);
#pragma unroll
        for (int i = 0; i < C::NB * C::TERMS; ++i) landed(ot[i / C::TERMS][i % C::TERMS]);
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
          for (int h = 0; h < HPT; ++h) {
            o[nb][h] = ot[nb][C::TERMS - 1][h];
#pragma unroll
            for (int t = C::TERMS - 2; t >= 0; --t) o[nb][h] = ot[nb][t][h] + o[nb][h] * (1.f / C::kNext);
          }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(B(o_empty[cu.seg & 1]));
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
          if (h0 + h >= G) break;
          // a sum of 0: nothing counted, and O may hold anything
          const float r = l[h] == 0.f ? 0.f : whole ? vs / l[h] : vs;
#pragma unroll
          for (int nb = 0; nb < C::NB; ++nb) {
            if (row >= HD) break;
            const size_t at = (size_t)(h0 + h) * HD + 128 * nb + row;
            const float v = l[h] == 0.f ? 0.f : o[nb][h] * r;
            if (whole) a.o[orow * HD + at] = __float2bfloat16_rn(v);
            else piece[at] = v;
          }
          if (row == 0) {
            if (!whole) {
              piece[G * HD + h0 + h] = ref[h];
              piece[G * HD + G + h0 + h] = l[h];
            } else if (a.lse) {
              a.lse[orow + h0 + h] = (ref[h] + log2f(l[h])) * kLn2;  // -inf + log2(0) where nothing counts
            }
          }
        }
        if (!whole) {
          const long long ub = u0 + k - (cu.c - cu.s.c0);  // the unit of chunk c0 of (m, gg)
          const int i = np_mine++ & 1;
          pm[i] = cu.m;
          pgg[i] = cu.gg;
          pa[i] = owner(U, nct, ub);
          pst[i] = split_at(U, nct, pa[i]) == ub;
          pb[i] = owner(U, nct, ub + (cu.s.c1 - cu.s.c0) - 1);
        }
        first_seg = false;
        fresh = true;
      }
      if (!last) advance(a, cu);
      if (end) c_seg = cu.c;
    }

    // Split (request, kv head)s: count this CTA's pieces in; the CTA that brings the last one joins
    // them all, in order, and leaves the counter at zero.
    if (np_mine > 0) {
      __threadfence();
      bar_sync(3, kSoft);
      if (tid == 0) {
        for (int i = 0; i < np_mine; ++i) {
          const bool is_last = atomicAdd(a.ws + pa[i], 1u) == (unsigned)(pb[i] - pa[i]);
          if (is_last) a.ws[pa[i]] = 0u;
          s_last[i] = is_last;
        }
        __threadfence();
      }
      bar_sync(3, kSoft);
      for (int i = 0; i < np_mine; ++i) {
        if (!s_last[i]) continue;
        const size_t orow = (size_t)pm[i] * a.n_q + (size_t)pgg[i] * G;
        // CTA j's piece is its first one (slot 2 j), but that of the CTA the (request, kv head) starts
        // in only if that CTA's run starts with it
        auto piece_of = [&](int j) { return part + (size_t)(2 * j + (j == pa[i] && !pst[i] ? 1 : 0)) * per_piece; };
        for (int e = 4 * tid; e < G * HD; e += 4 * kSoft) {
          const int hi = e / HD;
          float Mx = -INFINITY, Lx = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int j = pa[i]; j <= pb[i]; ++j) Mx = fmaxf(Mx, __ldcg(piece_of(j) + G * HD + hi));
#pragma unroll 8
          for (int j = pa[i]; j <= pb[i]; ++j) {
            const float* pc = piece_of(j);
            const float f = weight(__ldcg(pc + G * HD + hi), Mx);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(pc + e));
            Lx += __ldcg(pc + G * HD + G + hi) * f;
            v.x += x.x * f;
            v.y += x.y * f;
            v.z += x.z * f;
            v.w += x.w * f;
          }
          const float r = Lx == 0.f ? 0.f : 1.0f / Lx;
          *reinterpret_cast<uint2*>(a.o + orow * HD + e) =
              make_uint2(pack_bf16(v.x * r, v.y * r), pack_bf16(v.z * r, v.w * r));
          if (a.lse && e % HD == 0) a.lse[orow + hi] = (Mx + log2f(Lx)) * kLn2;
        }
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc::tc_fence_after();
    tc::tmem_relinquish();
    tc::tmem_dealloc(tmem, C::kCols);
  }
}

inline size_t piece_floats(int G, int hd) { return ((size_t)G * (hd + 2) + 3) / 4 * 4; }

int sm_count() {  // of the current device, asked for once
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 1;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int HD, bool FP8, int HPT>
cudaError_t launch(const PagedAttnArgs& a, const void* k_pages, const void* v_pages, cudaStream_t st) {
  using C = PCfg<HD, FP8>;
  EncodeTiled enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap tm[2];
  const int page = 1 << a.page_shift;
  for (int i = 0; i < 2; ++i) {  // the pages as rows of positions
    const cuuint64_t dims[2] = {(cuuint64_t)HD, (cuuint64_t)a.t * a.n_pages * (a.n_kv / a.t) * page};
    const cuuint64_t strides[1] = {(cuuint64_t)C::ROWB};
    const cuuint32_t box[2] = {(cuuint32_t)(C::INB / (FP8 ? 1 : 2)), (cuuint32_t)std::min(page, kP)}, es[2] = {1, 1};
    if (enc(&tm[i], FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(i ? v_pages : k_pages), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            C::INB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kernel = paged_attn_kernel<HD, FP8, HPT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sm_count(), kPagedMaxCtas);
  e = launch_dependent(kernel, dim3(grid), dim3(kThreads), C::SMEM, st, tm[0], tm[1], a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t paged_attn_workspace_bytes(int G, int hd) {
  return (kPagedMaxCtas + 2 * kPagedMaxCtas * piece_floats(G, hd)) * 4;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int kv_dtype, int hd, const void* k_pages, const void* v_pages,
                              cudaStream_t st) {
  auto go = [&](auto fp8) {
    constexpr bool F = decltype(fp8)::value;
    const bool few = a.n_q / a.n_kv <= 8;  // heads per kv head: 4 or 8 per softmax thread
    if (hd == 64) return few ? launch<64, F, 4>(a, k_pages, v_pages, st) : launch<64, F, 8>(a, k_pages, v_pages, st);
    if (hd == 128) return few ? launch<128, F, 4>(a, k_pages, v_pages, st) : launch<128, F, 8>(a, k_pages, v_pages, st);
    return few ? launch<256, F, 4>(a, k_pages, v_pages, st) : launch<256, F, 8>(a, k_pages, v_pages, st);
  };
  return kv_dtype == TP_BF16 ? go(std::false_type{}) : go(std::true_type{});
}

}  // namespace tpx
