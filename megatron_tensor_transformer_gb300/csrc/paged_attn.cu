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
// work is a list of (request, kv head)s, each a run of 128-position chunks after a fixed cost for its
// beginning and end, and is split evenly over the CTAs in order, so that one long request and many short
// ones load all SMs alike.  (Items handed out by a counter balanced the SMs better, whose shares of the
// HBM differ by 10%, but an item's look-up and joins cost more than that: 105 us against 89.8 for 131071
// tokens.)
// Both products run on tcgen05 with the cache as the 128-row operand, straight from where TMA put it:
//   S^T [128 positions, 16 heads] = K Q^T      K as it lies (rows of positions), Q padded to 16 heads
//   O^T [dims, 16 heads]         += V^T P^T    V as it lies too, read as the transposed operand
// so no byte of k or v passes through registers.  Two softmax teams take the chunks in turn, each with
// its own reference, sum and O^T (joined at the item's end), so one chunk's exponentials run beside the
// other's waits.  A thread holds one position and 4 or 8 heads; maxima are looked for across threads only
// when a score passes the step.
//   bf16 pages: P enters the product as two bf16 (its rounding and the rest), so that P's rounding
//     does not show beside the output's own; the tensor cores have the time.
//   e4m3 pages: e4m3 products (kind::f8f6f4).  q is split into two codes (q / 2^e = hi + lo, all of a
//     bf16's bits unless it is below 2^-10 of its head's largest value).  P is split into three, each the
//     rest of the one before times 16: good to 2^-11 of its value and 2^-25 of a weight of 1, so that
//     the many small weights of a long context are not lost.  The heads' scales go to the scores and to
//     the output.
// The codes of a split operand are columns of one MMA side by side (N = 16 per code) and their products
// are added when tensor memory is read: an MMA costs the 128-row operand's way out of shared memory,
// whatever N is, so a code more costs nothing and an MMA more does (62 cycles alone, 150 beside TMA's
// writes; one MMA per code took 120.8 us for 131071 tokens of the 70B heads).
// Warps: the softmax teams; a TMA producer (lane i looks up the page of box i and copies it: 16 to 64
// positions by 128 bytes); one issuing the scores' MMAs and one those of P V, each as soon as its operands are
// there (one thread for both made every chunk wait for the one before: 107.1 us instead of 95.5 for 131071
// tokens); one that walks the CTA's items (its part of a (request, kv head)) and brings their q.
// A (request, kv head) that is split over CTAs leaves a piece per CTA (sum of p v, ref, sum) in the workspace;
// the CTA that counts in last joins up to kFan of them in order, and the last of those joins these (one CTA
// joining 19 pieces took 10 us).  Every sum's order follows from the lengths and the SM count: runs repeat
// bit for bit.
// Measured on one GB300 (GPU time of a call among others, fractions of the measured copy's 6792 GB/s):
//   1 request of 131071 tokens, 64 q and 8 kv heads of 128, bf16, pages of 64        87.6 us, 90%
//   32 ragged requests up to 4096, the same heads, pages of 16                       53.4 us, 80%
//   256 ragged requests up to 700, the same heads, pages of 32                       86.2 us, 63%
//   48 ragged requests up to 8192, 128 q and 8 kv heads, e4m3, pages of 32           82.0 us, 66%
//   61 ragged requests, a window of 1024, 8 q and 4 kv heads of 256, pages of 128    43.0 us, 78%
//   1 request of 519 tokens, 32 q and 8 kv heads, pages of 16                        10.0 us (latency)
// What is left: the short request's chain, 3.1 us for a call without positions (launch, the lengths' sum), 3.9 more
// for one chunk (items, page look-up, copies, products, the row), 2.0 more once two chunks are joined; the ends of
// short requests and the SMs' unequal shares of the HBM; and over e4m3 each (request, kv head)'s beginning and end, 2.4
// us beside 0.7 us a chunk, with 16 heads per kv head 4.4 beside 0.79 (0.73 at the copy's rate).
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "paged.h"
#include "tc.h"
#include "tc_ptx.cuh"

namespace tpx {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoRef = -3.402823466e38f;  // no reference yet: fp32's lowest, which every finite score reaches (one
                                            // that only reaches it is rightly a weight of 1 under it)
constexpr int kP = 128;                    // positions per chunk: the rows of an MMA
constexpr int kN = 16;                     // heads of an MMA (its columns)
constexpr int kMasks = 32;                 // ring of the chunks' masks: above the chunks in flight
constexpr int kFan = 5;                    // pieces joined at once (131071 tokens: 87.4 us with 5, 89.2 with 8, 90.0 with 24)
constexpr int kSlots = 2 * kPagedMaxCtas;  // pieces: a split (request, kv head) is a CTA's first item or its last
constexpr int kWsHead = kPagedCounters;    // counters: by the slot of the first of kFan pieces, then of the first of all
static_assert(kWsHead == 2 * kSlots, "two counters per slot");

template <int HD, bool FP8>
struct PCfg {
  static constexpr int ROWB = HD * (FP8 ? 1 : 2);                 // bytes of a position
  static constexpr int INB = ROWB < 128 ? ROWB : 128;             // bytes of a box row
  static constexpr int NIB = ROWB / INB;                          // boxes side by side
  // Positions of a TMA box at most (a page's, if it has fewer): what lies outside the positions attended to is not
  // read beyond a box.  bf16 chunks of 32-position boxes came as fast as of 128, e4m3 ones only from 64 on.
  static constexpr int BOX = FP8 ? 64 : 32;
  static constexpr int STAGE = kP * ROWB;                         // k or v of a chunk
  static constexpr int NB = HD == 256 ? 2 : 1;                    // 128-dim blocks of O^T
  static constexpr int KS = FP8 ? 32 : 16;                        // k of an MMA
  static constexpr int TERMS = FP8 ? 3 : 2;                       // codes that P is split into
  static constexpr int PROW = kN * (FP8 ? 1 : 2);                 // bytes of a position of P
  static constexpr int PTILE = kP * PROW;
  static constexpr int QTERMS = FP8 ? 2 : 1;                      // codes of q, 16 rows each
  static constexpr int QBOX = QTERMS * kN * 128;                  // their rows' 128 bytes
  static constexpr int QTILE = (ROWB + 127) / 128 * QBOX;
  static constexpr int NS = std::min(16, 192 * 1024 / STAGE);     // stages, k and v in turn
  static constexpr float kStep = FP8 ? 1.f : 8.f;                 // ref may be behind the maximum by this
  static constexpr float kPLog = FP8 ? 7.f : 0.f;                 // weights are held times 2^this: up to 256 in e4m3
  static constexpr float kNext = FP8 ? 16.f : 1.f;                // each code of P after the first is held times this
  static constexpr int kUsed = 2 * kN * (QTERMS + 2 * NB * TERMS);  // TMEM: S [2][QTERMS][16], O [2][team][NB][TERMS][16]
  static constexpr uint32_t kCols = kUsed > 256 ? 512 : kUsed > 128 ? 256 : 128;
  static constexpr size_t kRing = (size_t)NS * STAGE;
  static constexpr size_t SMEM = kRing + 2 * TERMS * PTILE + 2 * QTILE;
  static_assert(NS >= 3, "a chunk's k and v and the next one's k");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// what a sum taken under reference m counts under the reference mx (0 where nothing was summed)
__device__ __forceinline__ float weight(float m, float mx) { return m == -INFINITY ? 0.f : ex2(m - mx); }

// the warp's largest value (a NaN is passed over)
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// The sums of v[0 .. N) over the warp: lane l gets that of v[l >> (5 - log2 N)].
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
  int o = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1, o >>= 1) {  // the upper half of the lanes takes the upper half of the sums
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = lane & o ? v[i + n] : v[i], give = lane & o ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(kFull, give, o);
    }
  }
  for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(kFull, v[0], o);
  return v[0];
}

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
__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t v) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3));
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t v) { return __half22float2(e4m3x2_half2(v)); }

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

// Units of a request's (request, kv head)s: `ends`, then two per chunk.
__device__ __forceinline__ int units_of(const Span& s, int ends) { return s.c0 == s.c1 ? 0 : ends + 2 * (s.c1 - s.c0); }
// CTA i of nct takes units [U i / nct, U (i + 1) / nct), nct at most U / 2; a chunk belongs to the CTA of its
// first unit, which is owner(u).
__device__ __forceinline__ long long quot(long long x, long long y) {  // x / y, both >= 0: a 64-bit division only if it must be
  return (x | y) >> 32 ? x / y : (long long)((uint32_t)x / (uint32_t)y);
}
__device__ __forceinline__ long long split_at(long long U, int nct, int i) { return quot(U * i, nct); }
__device__ __forceinline__ int owner(long long U, int nct, long long u) {
  return (int)quot((u + 1) * nct + U - 1, U) - 1;
}

// Chunks [c0, c1) of (m, gg), whose request attends to [lo, n): the piece of CTA blockIdx.x of those that CTAs
// a .. b leave in slots 2 a + second, 2 (a + 1), .., 2 b.  a == b: the whole of it.  m < 0: no more items.
struct __align__(16) Item {
  int m, gg, c0, c1, lo, n, a, b, second, pad[3];
};
// Bits of chunk c's 16-position groups with a position that counts: within [lo, n) and loaded.
__device__ __forceinline__ uint32_t group_bits(const Item& it, int c, uint32_t loaded) {
  const int a0 = max(0, it.lo - c * kP), a1 = min(kP, it.n - c * kP);
  return loaded & ((1u << ((a1 + 15) >> 4)) - 1) & ~((1u << (a0 >> 4)) - 1);
}
// A role's bounded waits.  After one that runs out (it sets the error word) the producer issues no more copies and
// the two issuing threads no more MMAs, and each waits, bounded again, for what it has in flight; the softmax warps
// go on without waiting to the item's end, so that their team's barriers are met.  Then the kernel ends: no copy
// lands in shared memory and no MMA in tensor memory that the CTA has given back.
// (The loop is a function of its own: inlined at every wait it made the roles' code together larger than the
// SM's instruction cache, and the kernel's time depend on where the compiler put what, by up to a quarter.)
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, unsigned* err, unsigned code) {
  const bool ok = tc::mbar_wait(bar, parity);
  if (!ok) atomicExch(err, code);
  return !ok;
}
struct Waits {
  unsigned* err;
  unsigned code;
  bool failed;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) {  // whether the phase is over
    if (tc::mbar_try_wait(bar, parity) || tc::mbar_try_wait(bar, parity)) return true;
    if (!failed) failed = wait_long(bar, parity, err, code);
    return !failed;
  }
};

// grid: one CTA per SM.  Softmax teams of NG groups of 4 warps; a group's threads hold HPT heads, NG HPT >= n_q / n_kv.
template <int HD, bool FP8, int HPT, int NG>
__global__ void __launch_bounds__(2 * NG * 128 + 128, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ PagedAttnArgs a) {
  using C = PCfg<HD, FP8>;
  constexpr int kTeam = NG * 128, kSoftWarps = 2 * NG * 4, kThreads = 2 * kTeam + 128, kWarps = kThreads / 32;
  // A chunk is two units of work, the beginning and end of a (request, kv head) kEnds.  bf16, 128 dims, with 1, 2, 3
  // and 4: 32 requests up to 4096 take 52.9, 53.1, 53.3 and 54.3 us, 100 up to 2000 74.9, 68.3, 68.6 and 69.2, 256
  // up to 700 91.6, 88.1, 84.6 and 84.4; 256 dims: 256 up to 700 63.7, 63.8, 64.8 and 66.3.  e4m3, 8 heads a thread,
  // with 6, 8, 10 and 12: 48 up to 8192 94.7, 91.4, 91.6 and 92.8, 100 up to 2000 88.8, 82.5, 80.0 and 79.7, 256 up to
  // 700 143.5, 140.5, 140.1 and 140.1, 32 up to 4096 42.5, 40.4, 40.7 and 40.6, 100 windows of 1024 78.1, 77.0, 75.1
  // and 74.8, 64 up to 512 37.8, 37.8, 37.6 and 38.0, long ones alike: 10 is the least over all of them.
  constexpr int kEnds = FP8 ? (HPT == 8 ? 10 : 6) : C::STAGE >= 64 * 1024 ? 1 : C::STAGE >= 32 * 1024 ? 3 : 4;
  constexpr int kProducer = kSoftWarps, kScores = kProducer + 1, kItems = kProducer + 2, kPV = kProducer + 3;
  extern __shared__ __align__(1024) uint8_t ring[];  // the swizzles' atoms; static shared memory is padded to it
  uint8_t* sQ = ring + C::kRing;           // [2][QTILE]
  uint8_t* sP = sQ + 2 * C::QTILE;         // [2][TERMS][PTILE], one per team
  __shared__ Item s_item[4];
  __shared__ __align__(8) uint64_t kv_full[2][C::NS], kv_empty[2][C::NS], q_full[2], q_empty[2], s_full[2], s_empty[2],
      p_full[2], p_empty[2], o_full[2], o_empty[2], x_full[2], x_empty[2], i_full[4], i_empty[4], mma_done[2];
  __shared__ long long s_part[kWarps], s_base;  // s_base: units before request s_m, which holds the CTA's first one
  __shared__ float s_max[kSoftWarps][HPT], s_sum[kSoftWarps][HPT], s_x[2][NG][2][HPT], q_pow[FP8 ? 4 : 1][kN];
  __shared__ uint32_t loaded[kMasks];                // 16-position groups of a chunk that were loaded, by bit
  __shared__ uint32_t s_tmem;
  __shared__ int s_last[2], s_m;
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
      tc::mbar_init(B(s_empty[i]), 4 * NG);
      tc::mbar_init(B(p_full[i]), 4 * NG);
      tc::mbar_init(B(p_empty[i]), 1);
      tc::mbar_init(B(o_full[i]), 1);
      tc::mbar_init(B(o_empty[i]), 4 * NG);
      tc::mbar_init(B(x_full[i]), NG);
      tc::mbar_init(B(x_empty[i]), 4 * NG);
      tc::mbar_init(B(mma_done[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(B(i_full[i]), 1);
      tc::mbar_init(B(i_empty[i]), kSoftWarps + 3);
    }
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  if (warp == kScores) tc::tmem_alloc(tc::smem_u32(&s_tmem), C::kCols);
  tc::griddep_wait();
  tc::griddep_launch_dependents();  // after the wait: what follows may then rely on all work before this kernel
  const int G = a.n_q / a.n_kv, nkvs = a.n_kv / a.t;

  // The units: a sum over the requests, a contiguous run of them per thread.
  const int per = (a.M + kThreads - 1) / kThreads, r0 = min(a.M, tid * per), r1 = min(a.M, r0 + per);
  long long here = 0;
  for (int m = r0; m < r1; ++m) here += (long long)units_of(span_of(a, m), kEnds) * a.n_kv;
  long long base = here;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(kFull, base, o);
    if (lane >= o) base += u;
  }
  if (lane == 31) s_part[warp] = base;
  base -= here;
  __syncthreads();
  long long U = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += s_part[w];
    U += s_part[w];
  }
  const int nct = (int)min((long long)gridDim.x, U / 2);
  const long long u0 = nct == 0 ? 0 : split_at(U, nct, min((int)blockIdx.x, nct)),
                  u1 = nct == 0 ? 0 : split_at(U, nct, min((int)blockIdx.x + 1, nct));
  if (u0 < u1 && u0 >= base && u0 < base + here) {  // this thread's requests hold unit u0
    int m = r0;
    for (;; ++m) {
      const long long n = (long long)units_of(span_of(a, m), kEnds) * a.n_kv;
      if (u0 < base + n) break;
      base += n;
    }
    s_m = m;
    s_base = base;
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto S_at = [&](int k, int term) { return tmem + ((k & 1) * C::QTERMS + term) * kN; };
  auto O_at = [&](int j, int team, int nb, int term) {
    return tmem + (2 * C::QTERMS + (((j & 1) * 2 + team) * C::NB + nb) * C::TERMS + term) * kN;
  };
  constexpr uint32_t kLay = C::INB == 128 ? 2 : 4;  // swizzle of the cache's stages
  auto mma = [](uint32_t d, uint64_t x, uint64_t y, uint32_t id, bool acc) {
    if (FP8) tc::mma_e4m3(d, x, y, id, acc);
    else tc::mma_bf16(d, x, y, id, acc);
  };
  // Item j as a role sees it: j counts the CTA's items, k its chunks (over all items) from here on.
  auto next_item = [&](Waits& wait, int j, bool whole_warp) {
    wait(B(i_full[j & 3]), (j >> 2) & 1);
    const Item it = s_item[j & 3];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) tc::mbar_arrive(B(i_empty[j & 3]));
    if (wait.failed) {  // nothing to go by: end
      Item none = it;
      none.m = -1;
      return none;
    }
    return it;
  };

  if (warp == kProducer) {
    // ---- k of chunk c in stage 2 c, v in 2 c + 1 (modulo NS).  The barriers go by (k or v, chunk modulo NS), not
    // by stage: each is then waited for phase by phase by one role (with an odd NS a stage holds k and v in
    // turn, and the role that reads k would miss every other phase).
    Waits wait{a.err, 44u, false};
    const int box_rows = min(1 << a.page_shift, C::BOX), nbp = kP / box_rows;  // boxes along the positions
    const int box = lane % nbp, side = lane / nbp;
    const uint64_t pol = tc::l2_evict_first();  // the cache streams through once
    // Page ids come 32 at a time, one per lane, the next 32 on their way (one chunk's at a time, a look-up
    // took as long as a chunk of 32 KB).
    auto first_page = [&](const Item& it) { return it.c0 * kP >> a.page_shift; };
    auto ids_from = [&](const Item& it, int page) {  // the page id of page + lane, -1: not attended to
      page += lane;
      const long long p = (long long)page << a.page_shift;
      return p < it.n && p + (1 << a.page_shift) > it.lo ? a.table[(size_t)it.m * a.table_stride + page] : -1;
    };
    int k = 0;
    bool stop = false;
    Item it = next_item(wait, 0, true), nx = it;
    int at = 0, ids = -1, ids_next = -1, ids_item = -1;  // lanes' ids from page `at` on; the 32 after; the next item's
    if (it.m >= 0) {
      at = first_page(it);
      ids = ids_from(it, at);
    }
    for (int j = 0; __all_sync(kFull, it.m >= 0) && !stop; ++j) {
      ids_next = ids_from(it, at + 32);
      auto look_ahead = [&]() {
        nx = next_item(wait, j + 1, true);
        if (nx.m >= 0) ids_item = ids_from(nx, first_page(nx));
      };
      const int base = (it.gg / nkvs) * a.n_pages, g = it.gg % nkvs;
      for (int c = it.c0; c < it.c1; ++c, ++k) {
        const int pos = c * kP + box * box_rows, page = pos >> a.page_shift;
        if (((c * kP + kP - 1) >> a.page_shift) >= at + 32) {  // a chunk's pages never straddle two batches
          at += 32;
          ids = ids_next;
          ids_next = ids_from(it, at + 32);
        }
        int id = __shfl_sync(kFull, ids, page - at);
        if (side >= C::NIB || pos >= it.n || pos + box_rows <= it.lo) id = -1;
        const bool load = id >= 0 && id < a.n_pages;
        const unsigned boxes = __ballot_sync(kFull, load);
        const unsigned groups = __ballot_sync(kFull, lane < 8 && (boxes >> ((lane & 7) * 16 / box_rows) & 1));
        const int row = (((base + id) * nkvs + g) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
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
        if (c == it.c0) look_ahead();
        // After a wait that ran out the chunk's copies are the last.  Their arrivals meet no open phase all the same:
        // copy i's barrier served copy i - 2 NS before, which the wait at copy i - NS has seen read.  (A vote before
        // the copies cost every stage 16 ns: e4m3 1 to 3%.)
        if (__any_sync(kFull, wait.failed)) {
          ++k;
          stop = true;
          break;
        }
      }
      it = nx;
      at = first_page(it);
      ids = ids_item;
    }
    static_assert(2 * C::NS <= 32, "a lane for every barrier");
    const int last = 2 * k - 1 - lane, lc = last >> 1;  // copies in flight: each barrier's last
    if (lane < 2 * C::NS && last >= 0) wait_long(B(kv_full[last & 1][lc % C::NS]), (lc / C::NS) & 1, a.err, 44u);
  } else if (warp == kScores) {
    // ---- scores: one thread issues
    if (lane == 0) {
      Waits wait{a.err, 45u, false};
      const uint32_t idesc = FP8 ? tc::idesc_e4m3(128, kN * C::QTERMS) : tc::idesc_bf16(128, kN * C::QTERMS);
      int k = 0;
      for (int j = 0;; ++j) {
        const Item it = next_item(wait, j, false);
        if (it.m < 0) break;
        if (!wait(B(q_full[j & 1]), (j >> 1) & 1)) break;
        const uint32_t qA = tc::smem_u32(sQ + (size_t)(j & 1) * C::QTILE);
        for (int c = it.c0; c < it.c1; ++c, ++k) {
          if (!wait(B(kv_full[0][k % C::NS]), (k / C::NS) & 1)) goto scores_end;
          if (k >= 2 && !wait(B(s_empty[k & 1]), ((k >> 1) - 1) & 1)) goto scores_end;
          tc::tc_fence_after();
          const uint32_t kA = tc::smem_u32(ring + (size_t)(2 * k % C::NS) * C::STAGE);
#pragma unroll
          for (int i = 0; i < C::ROWB / 32; ++i) {  // 32 bytes of a row per MMA
            const uint32_t ka = kA + (32 * i) / C::INB * (kP * C::INB) + (32 * i) % C::INB;
            const uint32_t qa = qA + i / 4 * C::QBOX + (i % 4) * 32;
            mma(S_at(k, 0), smem_desc(ka, 16, 8 * C::INB, kLay), smem_desc(qa, 16, 1024, 2), idesc, i > 0);
          }
          tc::mma_commit(B(kv_empty[0][k % C::NS]));
          tc::mma_commit(B(s_full[k & 1]));
          tc::mbar_arrive(B(s_full[k & 1]));  // releases what this thread has seen: the chunk's mask, q's powers
        }
        tc::mma_commit(B(q_empty[j & 1]));
      }
    scores_end:;
    }
    __syncwarp();
  } else if (warp == kPV) {
    // ---- P V: one thread issues.  The warp writes the rows without positions first, while the others begin.
    for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
      const Span s = span_of(a, m);
      if (s.c0 != s.c1) continue;
      uint4* o = reinterpret_cast<uint4*>(a.o + (size_t)m * a.n_q * HD);
      for (int i = lane; i < a.n_q * HD / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int i = lane; i < a.n_q; i += 32) a.lse[(size_t)m * a.n_q + i] = -INFINITY;
    }
    if (lane == 0) {
      Waits wait{a.err, 48u, false};
      const uint32_t idesc =
          (FP8 ? tc::idesc_e4m3(128, kN * C::TERMS) : tc::idesc_bf16(128, kN * C::TERMS)) | kTransposed;
      int k = 0;
      for (int j = 0;; ++j) {
        const Item it = next_item(wait, j, false);
        if (it.m < 0) break;
        if (j >= 2 && !wait(B(o_empty[j & 1]), ((j >> 1) - 1) & 1)) break;
        uint32_t live = 0;  // by team: its O holds something
        for (int c = it.c0; c < it.c1; ++c, ++k) {
          if (!wait(B(p_full[k & 1]), (k >> 1) & 1)) goto pv_end;
          if (!wait(B(kv_full[1][k % C::NS]), (k / C::NS) & 1)) goto pv_end;
          tc::tc_fence_after();
          const uint32_t groups = group_bits(it, c, loaded[k % kMasks]);
          const uint32_t vA = tc::smem_u32(ring + (size_t)((2 * k + 1) % C::NS) * C::STAGE);
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
              mma(O_at(j, k & 1, nb, 0), smem_desc(va, HD == 64 ? 0 : kP * C::INB, 8 * C::INB, kLay), pd, idesc,
                  live >> (k & 1) & 1);
            }
            live |= 1u << (k & 1);
          }
          tc::mma_commit(B(kv_empty[1][k % C::NS]));
          tc::mma_commit(B(p_empty[k & 1]));
        }
        tc::mma_commit(B(o_full[j & 1]));
      }
    pv_end:;
    }
    __syncwarp();
  } else if (warp == kItems) {
    // ---- items, and the q of each: G heads as 16 rows of 128-byte-swizzled pieces
    Waits wait{a.err, 46u, false};
    constexpr int RP = HD / 8;       // 16-byte pieces of a row: 8, 16 or 32 neighbouring lanes
    constexpr int QV = 16 * RP / 32;
    int m = u0 < u1 ? s_m : 0, gg = 0;
    Span s = u0 < u1 ? span_of(a, m) : Span{0, 0, 0, 0};
    long long at = u0 < u1 ? s_base : 0;  // the first unit of (m, gg)
    int j = 0;
    if (u0 < u1) {  // the head that holds u0
      const int n = units_of(s, kEnds);
      gg = (int)quot(u0 - at, n);
      at += (long long)gg * n;
    }
    for (;;) {
      Item it{};
      it.m = -1;
      if (__any_sync(kFull, wait.failed)) at = u1;  // for all lanes
      while (at < u1) {
        const int n = units_of(s, kEnds), ch = s.c1 - s.c0;
        if (n > 0) {
          // chunk i begins at unit at + kEnds + 2 i
          auto chunks_before = [&](long long u) {
            return (int)min((long long)ch, max(0ll, (u - at - kEnds + 1) >> 1));
          };
          it.c0 = chunks_before(u0);
          it.c1 = chunks_before(u1);
        }
        if (n > 0 && it.c0 < it.c1) {
          it.m = m;
          it.gg = gg;
          const bool split = it.c0 > 0 || it.c1 < ch;
          it.a = split ? owner(U, nct, at + kEnds) : 0;
          it.b = split ? owner(U, nct, at + kEnds + 2 * (ch - 1)) : 0;
          // whether it is the second item of CTA a, whose run then begins before it
          it.second = split && split_at(U, nct, it.a) < at;
          it.c0 += s.c0;
          it.c1 += s.c0;
          it.lo = s.lo;
          it.n = s.n;
        }
        at += n;
        if (++gg >= a.n_kv || n == 0) {
          gg = 0;
          if (++m >= a.M) at = u1;
          else s = span_of(a, m);
        }
        if (it.m >= 0) break;
      }
      if (j >= 4) wait(B(i_empty[j & 3]), ((j >> 2) - 1) & 1);
      if (lane == 0) {
        s_item[j & 3] = it;
        tc::mbar_arrive(B(i_full[j & 3]));
      }
      if (it.m < 0) break;
      const __nv_bfloat16* qp = a.q + ((size_t)it.m * a.n_q + (size_t)it.gg * G) * HD;
      uint4 qn[QV];
#pragma unroll
      for (int i = 0; i < QV; ++i) {
        const int idx = lane + 32 * i, r = idx / RP, c8 = idx % RP;
        qn[i] = r < G ? *reinterpret_cast<const uint4*>(qp + (size_t)r * HD + 8 * c8) : make_uint4(0, 0, 0, 0);
      }
      if (j >= 2) wait(B(q_empty[j & 1]), ((j >> 1) - 1) & 1);
      uint8_t* dst = sQ + (size_t)(j & 1) * C::QTILE;
#pragma unroll
      for (int i = 0; i < QV; ++i) {
        const int idx = lane + 32 * i, r = idx / RP, c8 = idx % RP;
        if (FP8) {  // q / 2^e below 256, as two codes
          const uint32_t w[4] = {qn[i].x, qn[i].y, qn[i].z, qn[i].w};
          uint32_t top = 0;
#pragma unroll
          for (int j2 = 0; j2 < 4; ++j2) top = max(top, max((w[j2] >> 7) & 0xffu, (w[j2] >> 23) & 0xffu));
#pragma unroll
          for (int o = 1; o < RP; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
          // exponent field of the largest value, less 7 for 2^7 <= q / 2^e < 2^8; both factors stay normal
          const int e = min(max((int)top, 8), 253) - 7;
          // an infinity would become the largest code: it makes the row NaN instead, as its scores would
          const float inv = top == 255u ? NAN : __uint_as_float((uint32_t)(254 - e) << 23);
          uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
          for (int j2 = 0; j2 < 4; ++j2) {
            const float v = bf16_lo(w[j2]) * inv, y = bf16_hi(w[j2]) * inv;
            const uint32_t h = e4m3x2(v, y);
            const float2 b = e4m3x2_value(h);
            hi[j2 >> 1] |= h << (16 * (j2 & 1));
            lo[j2 >> 1] |= e4m3x2(v - b.x, y - b.y) << (16 * (j2 & 1));
          }
          uint8_t* at = dst + c8 / 16 * C::QBOX + r * 128 + (((c8 / 2 % 8) ^ (r & 7)) << 4) + (c8 & 1) * 8;
          *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(at + kN * 128) = make_uint2(lo[0], lo[1]);
          if (c8 == 0) q_pow[j & 3][r] = __uint_as_float((uint32_t)e << 23);
        } else {
          *reinterpret_cast<uint4*>(dst + c8 / 8 * C::QBOX + r * 128 + (((c8 % 8) ^ (r & 7)) << 4)) = qn[i];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(B(q_full[j & 1]));
      ++j;
    }
  } else {
    // ---- softmax: thread = position 32 (warp % 4) + lane and heads [h0, h0 + HPT); for O, dim and heads.
    // Team k % 2 takes chunk k.
    Waits wait{a.err, 47u, false};
    const int team = warp / (4 * NG), grp = warp / 4 % NG, quad = warp & 3, h0 = grp * HPT, row = 32 * quad + lane;
    const int bid = 1 + team * NG + grp, tt = tid - team * kTeam;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    float* pieces = reinterpret_cast<float*>(a.ws + kWsHead);
    const int per_piece = (G * (HD + 2) + 3) / 4 * 4;
    int k0 = 0;  // chunks before the item
    for (int j = 0;; ++j) {
      const Item it = next_item(wait, j, true);
      // a team ends together: a thread whose wait has run out would leave the others at a barrier
      if (bar_any(5 + team, kTeam, it.m < 0)) break;
      const int nch = it.c1 - it.c0;
      // A weight is 2^(s sc - sub): sub = ref - kPLog, or kNoRef while there is no reference.
      float sub[HPT], l[HPT], sc[HPT];
#pragma unroll
      for (int h = 0; h < HPT; ++h) {
        sub[h] = kNoRef;
        l[h] = 0.f;
        sc[h] = a.scale * kLog2e * (FP8 && a.k_scale ? a.k_scale[it.gg] : 1.0f);
      }
      const float vs = FP8 && a.v_scale ? a.v_scale[it.gg] : 1.0f;
      bool live = false;  // O holds something
      const int first = (k0 ^ team) & 1;
      for (int i = first; i < nch; i += 2) {
        const int k = k0 + i, c = it.c0 + i;
        wait(B(s_full[team]), (k >> 1) & 1);
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
        if (FP8 && i == first) {
#pragma unroll
          for (int h = 0; h < HPT; ++h) sc[h] *= q_pow[j & 3][h0 + h];
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(B(s_empty[team]));
        const uint32_t groups = group_bits(it, c, loaded[k % kMasks]);
        const int p = c * kP + row;
        const bool counts = p >= it.lo && p < it.n && (groups >> (row >> 4) & 1);
        // The product is rounded by itself: the reference is such a product, and a fused difference from it would hold
        // its rounding, which passes every step once the scores' spacing does (from 2^25 on).
        float x[HPT], top = -INFINITY;
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
          s[h] = __fmul_rn(s[h], sc[h]);
          x[h] = counts ? s[h] - sub[h] : -INFINITY;
          top = fmaxf(top, x[h]);
        }
        const bool raise = bar_any(bid, 128, top > C::kStep + C::kPLog);
        if (k >= 2) wait(B(p_empty[team]), ((k >> 1) - 1) & 1);  // the team's P V before has ended
        if (raise) {  // a new reference: the maximum so far
#pragma unroll
          for (int h = 0; h < HPT; ++h) {
            float v = counts ? s[h] : -INFINITY;
            v = warp_max(v);
            if (lane == 0) s_max[warp][h] = v;
          }
          bar_sync(bid, 128);
          float f[HPT];
#pragma unroll
          for (int h = 0; h < HPT; ++h) {
            float v = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) v = fmaxf(v, s_max[(warp & ~3) + w][h]);
            const float to = fmaxf(sub[h], v - C::kPLog);  // kNoRef if there is still no score
            f[h] = ex2(sub[h] - to);                       // from kNoRef: of a sum that is 0
            l[h] *= f[h];
            sub[h] = to;
            x[h] = counts ? s[h] - sub[h] : -INFINITY;
          }
          if (live) {
            tc::tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < C::NB * C::TERMS; ++q) {
              const uint32_t at = O_at(j, team, q / C::TERMS, q % C::TERMS) + h0 + lanes;
              float o[HPT];
              tmem_ld<HPT>(at, o);
              landed(o);
#pragma unroll
              for (int h = 0; h < HPT; ++h) o[h] *= f[h];
              tmem_st<HPT>(at, o);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
          s[h] = ex2(x[h]);
          l[h] += s[h];
        }
        uint8_t* pt = sP + (size_t)team * C::TERMS * C::PTILE;
        if (FP8) {
          __half2 r[HPT / 2];  // good to 2^-11 of a weight, or 2^-32 of one that is 1
#pragma unroll
          for (int q = 0; q < HPT / 2; ++q) r[q] = __floats2half2_rn(s[2 * q], s[2 * q + 1]);
          const __half2 next = __float2half2_rn(C::kNext);
#pragma unroll
          for (int t = 0; t < C::TERMS; ++t) {
            uint32_t w[HPT / 4];
#pragma unroll
            for (int q = 0; q < HPT / 2; ++q) {
              const uint32_t code = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(r[q]), __NV_SATFINITE, __NV_E4M3);
              w[q >> 1] = q & 1 ? w[q >> 1] | code << 16 : code;
              if (t + 1 < C::TERMS) r[q] = __hmul2(__hsub2(r[q], e4m3x2_half2(code)), next);  // exact
            }
            uint8_t* at = pt + t * C::PTILE + row * 16 + h0;
            if constexpr (HPT == 8) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t*>(at) = w[0];
          }
        } else {
          uint32_t hi[HPT / 2], lo[HPT / 2];
#pragma unroll
          for (int q = 0; q < HPT / 2; ++q) {
            const float u = s[2 * q], y = s[2 * q + 1];
            hi[q] = pack_bf16(u, y);
            lo[q] = pack_bf16(u - bf16_lo(hi[q]), y - bf16_hi(hi[q]));
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
          wait(B(kv_full[1][k % C::NS]), (k / C::NS) & 1);
          if (step_runs && !counts) {
            constexpr int PB = C::INB / 16, NPC = C::ROWB / 16;  // a row's pieces stay within it under any swizzle
            uint8_t* v = ring + (size_t)((2 * k + 1) % C::NS) * C::STAGE + row * C::INB;
#pragma unroll
            for (int q = grp; q < NPC; q += NG)
              *reinterpret_cast<uint4*>(v + q / PB * (kP * C::INB) + (q % PB) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        live |= groups != 0;
        fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(B(p_full[team]));
      }

      // The item's end: the sums over the positions; the team of the first chunk brings the two together.
      s_sum[warp][lane / (32 / HPT)] = warp_sums(l, lane);  // (the same sum from each lane that has it)
      bar_sync(bid, 128);
#pragma unroll
      for (int h = 0; h < HPT; ++h) {
        const float(*q)[HPT] = &s_sum[warp & ~3];
        l[h] = (q[0][h] + q[1][h]) + (q[2][h] + q[3][h]);
      }
      k0 += nch;
      if (first != 0) {
        if (quad == 0 && lane == 0) {  // only who writes waits: another could come when the next phase has ended too
          if (j >= 2) wait(B(x_empty[j & 1]), ((j >> 1) - 1) & 1);
#pragma unroll
          for (int h = 0; h < HPT; ++h) {
            s_x[j & 1][grp][0][h] = sub[h];
            s_x[j & 1][grp][1][h] = l[h];
          }
          tc::mbar_arrive(B(x_full[j & 1]));
        }
        __syncwarp();
        continue;
      }
      wait(B(x_full[j & 1]), (j >> 1) & 1);
      float f0[HPT], f1[HPT];
#pragma unroll
      for (int h = 0; h < HPT; ++h) {
        const float xs = s_x[j & 1][grp][0][h], xl = s_x[j & 1][grp][1][h], v = fmaxf(sub[h], xs);
        // a sum of 0: nothing counted, and its O may hold anything
        f0[h] = l[h] == 0.f ? 0.f : ex2(sub[h] - v);
        f1[h] = xl == 0.f ? 0.f : ex2(xs - v);
        l[h] = l[h] * f0[h] + xl * f1[h];
        sub[h] = v;
      }
      wait(B(o_full[j & 1]), (j >> 1) & 1);
      tc::tc_fence_after();
      const bool whole = it.a == it.b;
      auto slot_of = [&](int cta) { return 2 * cta + (cta == it.a ? it.second : 0); };
      const size_t orow = (size_t)it.m * a.n_q + (size_t)it.gg * G;  // of o and lse
      float* piece = pieces + (size_t)slot_of(blockIdx.x) * per_piece;
#pragma unroll 1
      for (int nb = 0; nb < C::NB; ++nb) {
        float ot[2][C::TERMS][HPT];
#pragma unroll
        for (int q = 0; q < 2 * C::TERMS; ++q)
          tmem_ld<HPT>(O_at(j, team ^ (q / C::TERMS), nb, q % C::TERMS) + h0 + lanes, ot[q / C::TERMS][q % C::TERMS]);
#pragma unroll
        for (int q = 0; q < 2 * C::TERMS; ++q) landed(ot[q / C::TERMS][q % C::TERMS]);
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
          float v[2];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            v[w] = ot[w][C::TERMS - 1][h];
#pragma unroll
            for (int t = C::TERMS - 2; t >= 0; --t) v[w] = ot[w][t][h] + v[w] * (1.f / C::kNext);
          }
          const float r = !whole ? vs : l[h] == 0.f ? 0.f : __fdividef(vs, l[h]);
          const float o = ((f0[h] == 0.f ? 0.f : v[0] * f0[h]) + (f1[h] == 0.f ? 0.f : v[1] * f1[h])) * r;
          if (h0 + h < G && row < HD) {
            const size_t at = (size_t)(h0 + h) * HD + 128 * nb + row;
            if (whole) a.o[orow * HD + at] = __float2bfloat16_rn(o);
            else piece[at] = o;
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(B(o_empty[j & 1]));
        tc::mbar_arrive(B(x_empty[j & 1]));
      }
      if (row == 0) {
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
          if (h0 + h >= G) break;
          if (!whole) {
            piece[G * HD + h0 + h] = l[h] == 0.f ? -INFINITY : sub[h];
            piece[G * HD + G + h0 + h] = l[h];
          } else if (a.lse) {
            a.lse[orow + h0 + h] = l[h] == 0.f ? -INFINITY : (sub[h] + log2f(l[h])) * kLn2;
          }
        }
      }
      if (whole) continue;

      // A piece: count it in among kFan neighbours; who is last joins those pieces in order and counts in
      // among the joined ones, whose last gives the result.  The counters are left at zero.
      auto last_of = [&](unsigned* counter, int n) {  // whole team: its writes are seen by who is last
        bar_sync(5 + team, kTeam);
        if (tt == 0) {
          unsigned before;  // releases the team's writes, and acquires those of who counted in before
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
          const bool is_last = before + 1 == (unsigned)n;
          if (is_last) *counter = 0u;
          s_last[team] = is_last;
        }
        bar_sync(5 + team, kTeam);
        return s_last[team] != 0;
      };
      // the pieces of CTAs first, first + step, ..: n of them, in order
      auto join = [&](int e, size_t from, int cta0, int step, int n, float& M, float& L, float4& v) {
        const int hi = e / HD;
        M = -INFINITY;
        L = 0.f;
        v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b = 0; b < n; b += kFan) {
          float pm[kFan], pl[kFan];
          float4 pv[kFan];
          float Mb = M;
#pragma unroll
          for (int q = 0; q < kFan; ++q) {
            const float* pc = pieces + (from + slot_of(cta0 + min(b + q, n - 1) * step)) * per_piece;
            pm[q] = __ldcg(pc + G * HD + hi);
            pl[q] = __ldcg(pc + G * HD + G + hi);
            pv[q] = __ldcg(reinterpret_cast<const float4*>(pc + e));
          }
#pragma unroll
          for (int q = 0; q < kFan; ++q)
            if (b + q < n) Mb = fmaxf(Mb, pm[q]);
          const float g = weight(M, Mb);
          L *= g;
          v = make_float4(v.x * g, v.y * g, v.z * g, v.w * g);
#pragma unroll
          for (int q = 0; q < kFan; ++q) {
            if (b + q >= n) break;
            const float f = weight(pm[q], Mb);
            L += pl[q] == 0.f ? 0.f : pl[q] * f;
            v.x += pv[q].x * f;
            v.y += pv[q].y * f;
            v.z += pv[q].z * f;
            v.w += pv[q].w * f;
          }
          M = Mb;
        }
      };
      const int all = it.b - it.a + 1, fan0 = it.a + ((int)blockIdx.x - it.a) / kFan * kFan;
      const int nfan = min(kFan, it.b + 1 - fan0), nfans = (all + kFan - 1) / kFan;
      if (!last_of(a.ws + slot_of(fan0), nfan)) continue;
      int cta0 = fan0, step = 1, n = nfan;
      size_t from = 0;  // joined pieces lie kSlots behind the slot of their first
      for (bool final = nfans == 1;; final = true) {
#pragma unroll 1
        for (int e = 4 * tt; e < G * HD; e += 4 * kTeam) {
          float M, L;
          float4 v;
          join(e, from, cta0, step, n, M, L, v);
          if (!final) {
            float* dst = pieces + (kSlots + (size_t)slot_of(fan0)) * per_piece;
            *reinterpret_cast<float4*>(dst + e) = v;
            if (e % HD == 0) {
              dst[G * HD + e / HD] = M;
              dst[G * HD + G + e / HD] = L;
            }
            continue;
          }
          const float r = L == 0.f ? 0.f : 1.0f / L;
          *reinterpret_cast<uint2*>(a.o + orow * HD + e) =
              make_uint2(pack_bf16(v.x * r, v.y * r), pack_bf16(v.z * r, v.w * r));
          if (a.lse && e % HD == 0) a.lse[orow + e / HD] = (M + log2f(L)) * kLn2;
        }
        if (final || !last_of(a.ws + kSlots + slot_of(it.a), nfans)) break;
        cta0 = it.a;
        step = kFan;
        n = nfans;
        from = kSlots;
      }
    }
  }
  if ((warp == kScores || warp == kPV) && lane == 0) {  // its MMAs in flight
    tc::mma_commit(B(mma_done[warp == kPV]));
    wait_long(B(mma_done[warp == kPV]), 0, a.err, 49u);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kScores) {
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

template <int HD, bool FP8, int HPT, int NG>
cudaError_t launch(const PagedAttnArgs& a, const void* k_pages, const void* v_pages, cudaStream_t st) {
  using C = PCfg<HD, FP8>;
  EncodeTiled enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap tm[2];
  const int page = 1 << a.page_shift;
  for (int i = 0; i < 2; ++i) {  // the pages as rows of positions
    const cuuint64_t dims[2] = {(cuuint64_t)HD, (cuuint64_t)a.t * a.n_pages * (a.n_kv / a.t) * page};
    const cuuint64_t strides[1] = {(cuuint64_t)C::ROWB};
    const cuuint32_t box[2] = {(cuuint32_t)(C::INB / (FP8 ? 1 : 2)), (cuuint32_t)std::min(page, C::BOX)}, es[2] = {1, 1};
    if (enc(&tm[i], FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(i ? v_pages : k_pages), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            C::INB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kernel = paged_attn_kernel<HD, FP8, HPT, NG>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sm_count(), kPagedMaxCtas);
  e = launch_dependent(kernel, dim3(grid), dim3(2 * NG * 128 + 128), C::SMEM, st, tm[0], tm[1], a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t paged_attn_workspace_bytes(int G, int hd) {
  return (kWsHead + 2 * kSlots * piece_floats(G, hd)) * 4;  // the pieces, and the joined ones
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int kv_dtype, int hd, const void* k_pages, const void* v_pages,
                              cudaStream_t st) {
  auto go = [&](auto fp8) {
    constexpr bool F = decltype(fp8)::value;
    auto sized = [&](auto hd_) {
      constexpr int D = decltype(hd_)::value;
      const int G = a.n_q / a.n_kv;  // heads of a kv head: 4 or 8 per softmax thread, in one or two groups
      return G <= 4   ? launch<D, F, 4, 1>(a, k_pages, v_pages, st)
             : G <= 8 ? launch<D, F, 4, 2>(a, k_pages, v_pages, st)
                      : launch<D, F, 8, 2>(a, k_pages, v_pages, st);
    };
    if (hd == 64) return sized(std::integral_constant<int, 64>{});
    if (hd == 128) return sized(std::integral_constant<int, 128>{});
    return sized(std::integral_constant<int, 256>{});
  };
  return kv_dtype == TP_BF16 ? go(std::false_type{}) : go(std::true_type{});
}

}  // namespace tpx
