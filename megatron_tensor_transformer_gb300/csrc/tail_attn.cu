// What each request attends to by itself beside its group's shared prefix (prefix_attn.cu): often a few hundred
// positions of many requests.
//
// Per (request, kv head), up to 16 q heads as the rows of mma.sync products, over stages of 32 to 128 positions.  It is
// HBM-bound, and with short runs bound by the chain of a run's beginning and end: page look-up, copies, products, sums.  So
// two or three small CTAs share an SM, whose chains overlap, in place of one with many roles.  A CTA takes an even share of all
// stages: one warp walks them, looks up pages, issues the TMA copies and brings the q of each run, four compute.
//
// Both products permute their summed index, so that a thread's operands lie side by side: for the scores a thread
// takes 16 bytes of each key's row (8 dims, or 16 of e4m3) and the same dims of q; for P V positions are taken as the
// scores left them.  Weights enter the product as two bf16, their rounding and the rest (2^-16 of a weight, so that it does
// not show beside the output's own rounding; the tensor cores have the time), or as fp16 over e4m3 pages, whose codes become
// fp16 in registers (exact).  Scores of positions that are not attended to are -inf, and their v is zeroed in shared memory.
//
// Measured (one launch, cold): 2048 runs of up to 250 positions (194 MB) 47 us, 4.1 TB/s; runs that take 71 MB 26 us, 2.8 TB/s,
// 10 us of which pass before the first product; one bf16 for a weight instead of two takes no less.  With the paged kernel's
// CTAs in its place a batch of the latter took 69 us in all.  Long runs take more here than there: 16 requests of up to 30000
// positions that share nothing 159 us for a call, 144 as paged attention (e4m3 98 and 81).
#include <cuda.h>

#include <algorithm>

#include "paged_attn.cuh"
#include "tc.h"

namespace tpx {

namespace {

template <int HD, bool FP8>
struct TCfg {
  static constexpr int ROWB = HD * (FP8 ? 1 : 2);              // bytes of a position
  static constexpr int INB = ROWB < 128 ? ROWB : 128;          // bytes of a box row
  static constexpr int NIB = ROWB / INB;                       // boxes side by side
  static constexpr int SP = tail_positions(HD, FP8);           // positions per stage
  static constexpr int BOX = SP < 32 ? SP : 32;                // of a TMA box at most: beyond a run's ends less is read
  static constexpr int SIDE = SP * ROWB;                       // k or v of a stage
  static constexpr int WD = HD == 256 ? 2 : 1, WP = 4 / WD;    // warps along v's dims and along the positions
  static constexpr int NBK = SP / (16 * WP);                   // blocks of 16 positions per warp
  static constexpr int ND = HD / WD / 8;                       // 8-dim blocks of O per warp
  static constexpr int QROW = HD * 2 + 16;                     // bytes of a row of q
  static constexpr int kJoin = WP * 16 * HD * 4;               // the warps' sums at a run's end
  static constexpr int STAGE = std::max(2 * SIDE, kJoin);      // they lie in the stage that was computed on last
  static constexpr int NST = 2;
  static constexpr int SMEM = NST * STAGE + 2 * 16 * QROW;
  static constexpr float kPLog = FP8 ? 7.f : 0.f;              // weights are held times 2^this
  static constexpr int kPerSm = HD == 256 ? 2 : 3;             // CTAs that an SM holds
  static_assert(kPerSm * (SMEM + (3 << 10)) <= 228 * 1024, "shared memory of an SM");
  static_assert(STAGE % 1024 == 0, "swizzle atoms");
};
constexpr int kCompute = 128, kThreads = kCompute + 32;

// 16-byte piece u of row r of a stage's k or v, as TMA swizzles it
template <int HD, bool FP8>
__device__ __forceinline__ int at_of(int r, int u) {
  using C = TCfg<HD, FP8>;
  if (C::INB == 64) return r * 64 + ((u ^ (r >> 1 & 3)) << 4);
  return (u >> 3) * (C::SP * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4);
}

template <bool FP8>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (!FP8) {
    mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
__device__ __forceinline__ uint32_t half2_of(uint32_t codes) {  // the low two
  const __half2 x = e4m3x2_half2(codes & 0xffffu);
  return *reinterpret_cast<const uint32_t*>(&x);
}

__device__ __forceinline__ void bar_compute() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool bar_compute_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

// A stage of a run: positions [c SP, c SP + SP) of (m, gg), of [lo, n).
struct Step {
  int m, gg, c, c1;    // c1: the end of this CTA's part of the run.  m < 0: no more
  int lo, n, first, ch;  // first: c is its part's first; ch: stages of the whole run, from lo / SP on
  long long at;        // the run's first unit
};
// What the computing warps need of it.
struct __align__(16) Desc {
  int m, gg, p0, lo;  // p0: the stage's first position
  int n, flags;       // kFirst, kLast, kWhole, kSecond, kQ: the buffer of q
  uint32_t in;        // 16-position groups that were loaded, by bit
  int pad;
};
constexpr int kFirst = 1, kLast = 2, kWhole = 4, kSecond = 8, kQ = 16;

template <int HD, bool FP8>
__global__ void __launch_bounds__(kThreads, TCfg<HD, FP8>::kPerSm)
    tail_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ GroupedAttnArgs a) {
  using C = TCfg<HD, FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem + C::NST * C::STAGE;  // [2][16][QROW]
  __shared__ __align__(8) uint64_t full[C::NST], empty[C::NST];
  __shared__ Desc s_desc[C::NST];
  __shared__ long long s_part[kThreads / 32], s_base;
  __shared__ float s_ref[C::WP][16], s_sum[C::WP][16], q_pow[2][16];
  __shared__ int s_m;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto B = [](const uint64_t& b) { return tc::smem_u32(&b); };
  if (tid == 0) {
    for (int i = 0; i < C::NST; ++i) {
      tc::mbar_init(B(full[i]), 1);
      tc::mbar_init(B(empty[i]), 4);
    }
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  // No wait for the kernel before: it began after all work before the call, so that this one did too, and this one reads
  // nothing of its.  At the end it is waited for, so that what follows this kernel follows both.
  tc::griddep_launch_dependents();
  const int G = a.n_q / a.n_kv;
  const bool groups = __syncthreads_and(groups_in_order(a, tid, kThreads));

  // The units: kTailEnds for a run's beginning and end and one per stage; a contiguous run of requests per thread.
  auto span = [&](int m) { return own_span<C::SP>(a, m, groups); };
  auto units = [&](const Span& s) { return s.c0 == s.c1 ? 0 : kTailEnds + (s.c1 - s.c0); };
  const int per = (a.M + kThreads - 1) / kThreads, r0 = min(a.M, tid * per), r1 = min(a.M, r0 + per);
  long long here = 0;
  for (int m = r0; m < r1; ++m) here += (long long)units(span(m)) * a.n_kv;
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
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += s_part[w];
    U += s_part[w];
  }
  const int nct = (int)min((long long)gridDim.x, U);
  const long long u0 = nct == 0 ? 0 : quot_call(U * min((int)blockIdx.x, nct), nct),
                  u1 = nct == 0 ? 0 : quot_call(U * min((int)blockIdx.x + 1, nct), nct);
  if (blockIdx.x == 0) {  // for the join
    if (tid == 0) {
      a.own_plan[0] = U;
      a.own_plan[1] = nct;
    }
    long long at = base;
    for (int m = r0; m < r1; ++m) {
      a.own_plan[2 + m] = at;
      at += (long long)units(span(m)) * a.n_kv;
    }
  }
  if (u0 < u1 && u0 >= base && u0 < base + here) {  // this thread's requests hold unit u0
    int m = r0;
    for (;; ++m) {
      const long long n = (long long)units(span(m)) * a.n_kv;
      if (u0 < base + n) break;
      base += n;
    }
    s_m = m;
    s_base = base;
  }
  __syncthreads();

  if (warp == 4) {
    // ---- the stages in order: page ids, copies, the q of each run
    const int nkvs = a.n_kv / a.t;
    const int box_rows = min(1 << a.page_shift, C::BOX), nb = C::SP / box_rows, box = lane % nb, side = lane / nb;
    int wm = 0, wg = 0;
    Span ws{0, 0, 0, 0};
    long long wat = u1;  // the first unit of (wm, wg)
    if (u0 < u1) {
      wm = s_m;
      ws = span(wm);
      const int n = units(ws);
      wg = (int)quot_call(u0 - s_base, n);
      wat = s_base + (long long)wg * n;
    }
    Step last{};
    last.m = -1;
    auto advance = [&]() {
      if (last.c + 1 < last.c1) {
        ++last.c;
        last.first = 0;
        return last;
      }
      last.m = -1;
      last.c1 = 0;
      while (wat < u1) {
        const int n = units(ws), ch = ws.c1 - ws.c0;
        if (n > 0) {
          // stage i is unit wat + kTailEnds + i
          const int c0 = (int)min((long long)ch, max(0ll, u0 - wat - kTailEnds)),
                    c1 = (int)min((long long)ch, max(0ll, u1 - wat - kTailEnds));
          if (c0 < c1) last = Step{wm, wg, ws.c0 + c0, ws.c0 + c1, ws.lo, ws.n, 1, ch, wat};
        }
        wat += n;
        if (++wg >= a.n_kv || n == 0) {
          wg = 0;
          if (++wm >= a.M) wat = u1;
          else ws = span(wm);
        }
        if (last.c1 > 0) break;
      }
      return last;
    };
    auto id_of = [&](const Step& s) {  // of the lane's box, -1: not attended to
      const int p = s.c * C::SP + box * box_rows;
      return s.m >= 0 && side < C::NIB && p < s.n && p + box_rows > s.lo
                 ? a.table[(size_t)s.m * a.table_stride + (p >> a.page_shift)]
                 : -1;
    };
    constexpr int RP = HD / 8, QV = 16 * RP / 32;  // 16-byte pieces of a row of q, of a lane
    uint4 qn[QV];
    auto load_q = [&](const Step& s) {
      const __nv_bfloat16* q = a.q + ((size_t)s.m * a.n_q + (size_t)s.gg * G) * HD;
#pragma unroll
      for (int i = 0; i < QV; ++i) {
        const int r = (lane + 32 * i) / RP, c8 = (lane + 32 * i) % RP;
        qn[i] = r < G ? *reinterpret_cast<const uint4*>(q + (size_t)r * HD + 8 * c8) : make_uint4(0, 0, 0, 0);
      }
    };
    auto store_q = [&](int buf) {
#pragma unroll
      for (int i = 0; i < QV; ++i) {
        const int r = (lane + 32 * i) / RP, c8 = (lane + 32 * i) % RP;
        uint8_t* dst = sQ + (buf * 16 + r) * C::QROW + 16 * c8;
        if (FP8) {
          int e;
          *reinterpret_cast<uint4*>(dst) = q_as_fp16<RP>(qn[i], e);
          if (c8 == 0) q_pow[buf][r] = __uint_as_float((uint32_t)e << 23);
        } else {
          *reinterpret_cast<uint4*>(dst) = qn[i];
        }
      }
    };
    const uint64_t pol = tc::l2_evict_first();  // read once
    Step cur = advance();
    int id = id_of(cur), run = -1;
    bool failed = false;
    int s = 0;
    for (;; ++s) {
      if (cur.m >= 0 && cur.first) {
        load_q(cur);
        ++run;
      }
      const Step nxt = cur.m >= 0 ? advance() : cur;
      const int id_next = id_of(nxt);
      const int st = s % C::NST;
      if (s >= C::NST && !tc::mbar_wait(B(empty[st]), (s / C::NST - 1) & 1)) {
        atomicExch(a.err, 60u);
        failed = true;
      }
      if (__any_sync(kFull, failed)) break;
      const bool load = id >= 0 && id < a.n_pages;
      const unsigned boxes = __ballot_sync(kFull, load);
      const unsigned in = __ballot_sync(kFull, lane < C::SP / 16 && (boxes >> ((lane * 16 / box_rows) & 31) & 1));
      if (lane == 0) tc::mbar_expect_tx(B(full[st]), 2 * __popc(boxes) * box_rows * C::INB);
      __syncwarp();
      if (load) {
        const int p = cur.c * C::SP + box * box_rows;
        const int row = ((((cur.gg / nkvs) * a.n_pages + id) * nkvs + cur.gg % nkvs) << a.page_shift) +
                        (p & ((1 << a.page_shift) - 1));
        const uint32_t dst = tc::smem_u32(smem + st * C::STAGE) + (side * C::SP + box * box_rows) * C::INB;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
          tc::tma_load_2d_hint(dst + kv * C::SIDE, kv ? &tmV : &tmK, side * (C::INB / (FP8 ? 1 : 2)), row, B(full[st]), pol);
      }
      if (cur.m >= 0 && cur.first) store_q(run & 1);  // beside the copies
      __syncwarp();
      if (lane == 0) {
        Desc d{cur.m, cur.gg, cur.c * C::SP, cur.lo, cur.n, 0, in, 0};
        if (cur.m >= 0) {
          d.flags = (cur.first ? kFirst : 0) | (run & 1 ? kQ : 0);
          if (cur.c + 1 == cur.c1) {
            // the run's first stage is this CTA's, and its last one: all of it; a piece is the CTA's second where it
            // begins the run, and the CTA's list begins before
            const bool begins = u0 <= cur.at + kTailEnds, ends = u1 >= cur.at + kTailEnds + cur.ch;
            d.flags |= kLast | (begins && ends ? kWhole : 0) | (begins && u0 < cur.at ? kSecond : 0);
          }
        }
        s_desc[st] = d;
        tc::mbar_arrive(B(full[st]));
      }
      if (cur.m < 0) {
        ++s;
        break;
      }
      cur = nxt;
      id = id_next;
    }
    const int mine = s - 1 - lane;  // copies in flight: each stage's last
    if (lane < C::NST && mine >= 0 && !tc::mbar_wait(B(full[mine % C::NST]), (mine / C::NST) & 1)) atomicExch(a.err, 60u);
  } else {
    // ---- four warps compute
    const int g8 = lane >> 2, t4 = lane & 3, wp = warp % C::WP, wd = warp / C::WP;
    float o[C::ND][4], m2[2], l2[2];  // rows g8 and g8 + 8: the reference (less kPLog) and the thread's part of the sum
    const float sc0 = a.scale * kLog2e;
    float sc[2] = {sc0, sc0};
    // Column c of tile t of a block's scores is this row of the block: bf16, so that the rows that a scores' load
    // takes together lie 4 apart (in other banks).
    auto row_of = [](int c, int t) { return (FP8 ? c : (c >> 1) + 4 * (c & 1)) + 8 * t; };
    const int p0 = 16 * C::NBK * wp;  // the warp's first position of a stage
    for (int st_n = 0;; ++st_n) {
      const int st = st_n % C::NST;
      const bool late = !tc::mbar_wait(B(full[st]), (st_n / C::NST) & 1);
      if (late) atomicExch(a.err, 61u);
      if (bar_compute_any(late)) break;  // together: they meet at barriers
      const Desc d = s_desc[st];
      if (d.m < 0) break;
      uint8_t *sK = smem + st * C::STAGE, *sV = sK + C::SIDE;
      const uint8_t* q0 = sQ + (d.flags & kQ ? 16 * C::QROW : 0) + g8 * C::QROW;
      if (d.flags & kFirst) {
#pragma unroll
        for (int i = 0; i < C::ND; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
        m2[0] = m2[1] = kNoRef;
        l2[0] = l2[1] = 0.f;
        if (FP8) {
          const float ks = a.k_scale ? a.k_scale[d.gg] : 1.f;
          const float* pow = q_pow[d.flags & kQ ? 1 : 0];
          sc[0] = sc0 * ks * pow[g8];
          sc[1] = sc0 * ks * pow[g8 + 8];
        }
      }
      // whether the stage's row r counts
      auto counts = [&](int r) { return (d.in >> (r >> 4) & 1) && d.p0 + r >= d.lo && d.p0 + r < d.n; };
      const bool edge = d.p0 + p0 < d.lo || d.p0 + p0 + 16 * C::NBK > d.n ||
                        (~d.in >> (p0 >> 4) & ((1u << C::NBK) - 1)) != 0;  // not all of the warp's rows do
      if (edge) {  // their v may be anything, NaN too
        constexpr int kUnits = C::ROWB / 16 / C::WD;
#pragma unroll 1
        for (int i = lane; i < 16 * C::NBK * kUnits; i += 32) {
          const int r = p0 + i / kUnits;
          if (!counts(r)) *reinterpret_cast<uint4*>(sV + at_of<HD, FP8>(r, wd * kUnits + i % kUnits)) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }

      // the scores of the warp's positions: [16 heads, 16 positions] per block, two tiles of 8 columns
      float s[C::NBK][2][4];
#pragma unroll
      for (int b = 0; b < C::NBK; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[b][t][k] = 0.f;
#pragma unroll
      for (int kb = 0; kb < C::ROWB / 64; ++kb) {  // 64 bytes of a row, 16 per thread
        constexpr int kSteps = FP8 ? 4 : 2;        // of 16 dims: 4 per thread
        uint32_t qa[kSteps][4];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint8_t* q = q0 + (FP8 ? 128 : 64) * kb + (FP8 ? 32 : 16) * t4 + 8 * i;
          const uint2 x = *reinterpret_cast<const uint2*>(q), y = *reinterpret_cast<const uint2*>(q + 8 * C::QROW);
          qa[i][0] = x.x;
          qa[i][1] = y.x;
          qa[i][2] = x.y;
          qa[i][3] = y.y;
        }
#pragma unroll
        for (int b = 0; b < C::NBK; ++b)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint4 k = *reinterpret_cast<const uint4*>(sK + at_of<HD, FP8>(p0 + 16 * b + row_of(g8, t), 4 * kb + t4));
            const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              if (FP8) mma16<true>(s[b][t], qa[i], half2_of(w[i]), half2_of(w[i] >> 16));
              else mma16<false>(s[b][t], qa[i], w[2 * i], w[2 * i + 1]);
            }
          }
      }
      // a running reference per warp and row; the product is rounded by itself, so that equal scores weigh the same
      float top[2] = {m2[0] + C::kPLog, m2[1] + C::kPLog};
#pragma unroll
      for (int b = 0; b < C::NBK; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[b][t][k] = __fmul_rn(s[b][t][k], sc[k >> 1]);
            if (edge && !counts(p0 + 16 * b + row_of(2 * t4 + (k & 1), t))) s[b][t][k] = -INFINITY;
            top[k >> 1] = fmaxf(top[k >> 1], s[b][t][k]);
          }
      bool grew = false;
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
        const float to = fmaxf(m2[h], top[h] - C::kPLog);
        grew |= to != m2[h];
        f[h] = ex2(m2[h] - to);
        m2[h] = to;
        l2[h] *= f[h];
      }
      if (__any_sync(kFull, grew)) {
#pragma unroll
        for (int i = 0; i < C::ND; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][k] *= f[k >> 1];
      }
#pragma unroll
      for (int b = 0; b < C::NBK; ++b) {
        uint32_t pa[4], pb[4];  // over bf16 pages a weight is two bf16, the second what the first leaves
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x = ex2(s[b][t][2 * h] - m2[h]), y = ex2(s[b][t][2 * h + 1] - m2[h]);
            l2[h] += x + y;
            if (FP8) {
              const __half2 z = __floats2half2_rn(x, y);
              pa[2 * t + h] = *reinterpret_cast<const uint32_t*>(&z);
            } else {
              pa[2 * t + h] = pack_bf16(x, y);
              pb[2 * t + h] = pack_bf16(x - bf16_lo(pa[2 * t + h]), y - bf16_hi(pa[2 * t + h]));
            }
          }
        if (FP8) {
          // 32 dims at a time, dim 4 c + j being column c of tile j: 4 positions by 4 dims per thread, turned
#pragma unroll
          for (int e = 0; e < C::ND / 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int byte = (HD / C::WD) * wd + 32 * e + 4 * g8;
              w[i] = *reinterpret_cast<const uint32_t*>(
                  sV + at_of<HD, FP8>(p0 + 16 * b + row_of(2 * t4 + (i & 1), i >> 1), byte >> 4) + (byte & 15));
            }
            const uint32_t x0 = __byte_perm(w[0], w[1], 0x5140), x1 = __byte_perm(w[0], w[1], 0x7362),
                           y0 = __byte_perm(w[2], w[3], 0x5140), y1 = __byte_perm(w[2], w[3], 0x7362);
            mma16<true>(o[4 * e], pa, half2_of(x0), half2_of(y0));
            mma16<true>(o[4 * e + 1], pa, half2_of(x0 >> 16), half2_of(y0 >> 16));
            mma16<true>(o[4 * e + 2], pa, half2_of(x1), half2_of(y1));
            mma16<true>(o[4 * e + 3], pa, half2_of(x1 >> 16), half2_of(y1 >> 16));
          }
        } else {
          // two tiles of 8 dims at a time; matrix row i of a tile's half t is row_of(i, t)
#pragma unroll
          for (int e = 0; e < C::ND; e += 2) {
            const int i = lane & 7, t = lane >> 3 & 1, u = (HD / C::WD) * wd / 8 + e + (lane >> 4);
            uint32_t v[4];
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(tc::smem_u32(sV) + at_of<HD, FP8>(p0 + 16 * b + row_of(i, t), u))
                         : "memory");
            mma16<false>(o[e], pa, v[0], v[1]);
            mma16<false>(o[e + 1], pa, v[2], v[3]);
            mma16<false>(o[e], pb, v[0], v[1]);
            mma16<false>(o[e + 1], pb, v[2], v[3]);
          }
        }
      }

      if (d.flags & kLast) {
        // The run's end: the warps' sums under their largest reference, added in order, to the joining kernel.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          l2[h] += __shfl_xor_sync(kFull, l2[h], 1);
          l2[h] += __shfl_xor_sync(kFull, l2[h], 2);
          if (t4 == 0 && wd == 0) {
            s_ref[wp][g8 + 8 * h] = m2[h];
            s_sum[wp][g8 + 8 * h] = l2[h];
          }
        }
        bar_compute();  // and all have read the stage
        float* slab = reinterpret_cast<float*>(sK) + wp * 16 * HD;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = g8 + 8 * h;
          if (row >= G) continue;
          float ref = s_ref[0][row];
#pragma unroll
          for (int w = 1; w < C::WP; ++w) ref = fmaxf(ref, s_ref[w][row]);
          const float fw = ex2(m2[h] - ref);  // a sum of 0 stays 0: its products' operands are zeros or finite
#pragma unroll
          for (int i = 0; i < C::ND; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int col = FP8 ? 32 * (i >> 2) + 4 * (2 * t4 + k) + (i & 3) : 8 * i + 2 * t4 + k;
              slab[row * HD + (HD / C::WD) * wd + col] = o[i][2 * h + k] * fw;
            }
        }
        bar_compute();
        const float vs = FP8 && a.v_scale ? a.v_scale[d.gg] : 1.f;
        const bool whole = d.flags & kWhole;
        const size_t row0 = (size_t)d.m * a.n_q + (size_t)d.gg * G;
        float* piece = a.own_pieces + (size_t)(2 * blockIdx.x + (d.flags & kSecond ? 1 : 0)) * a.own_piece;
        float* dst = whole ? a.part_o + row0 * HD : piece;
        for (int e = 4 * tid; e < G * HD; e += 4 * kCompute) {
          const float* src = reinterpret_cast<const float*>(sK) + e;
          float4 v = *reinterpret_cast<const float4*>(src);
#pragma unroll
          for (int w = 1; w < C::WP; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(src + w * 16 * HD);
            v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
          }
          *reinterpret_cast<float4*>(dst + e) = make_float4(v.x * vs, v.y * vs, v.z * vs, v.w * vs);
        }
        if (tid < G) {
          float ref = s_ref[0][tid], sum = 0.f;
#pragma unroll
          for (int w = 1; w < C::WP; ++w) ref = fmaxf(ref, s_ref[w][tid]);
#pragma unroll
          for (int w = 0; w < C::WP; ++w) sum += s_sum[w][tid] * ex2(s_ref[w][tid] - ref);
          (whole ? a.part_ref + row0 : piece + G * HD)[tid] = ref;
          (whole ? a.part_l + row0 : piece + G * HD + G)[tid] = sum;
        }
      }
      if (edge || (d.flags & kLast)) fence_proxy_async_smem();  // the stage was written here; TMA writes it next
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(B(empty[st]));
    }
  }
  __syncthreads();
  tc::griddep_wait();
}

template <int HD, bool FP8>
cudaError_t launch(const GroupedAttnArgs& a, cudaStream_t st) {
  using C = TCfg<HD, FP8>;
  EncodeTiled enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const int page = 1 << a.page_shift;
  CUtensorMap tm[2];
  for (int i = 0; i < 2; ++i) {  // the pages as rows of positions
    const cuuint64_t dims[2] = {(cuuint64_t)HD, (cuuint64_t)a.t * a.n_pages * (a.n_kv / a.t) * page};
    const cuuint64_t strides[1] = {(cuuint64_t)C::ROWB};
    const cuuint32_t box[2] = {(cuuint32_t)(C::INB / (FP8 ? 1 : 2)), (cuuint32_t)std::min(page, C::BOX)}, es[2] = {1, 1};
    if (enc(&tm[i], FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<uint8_t*>(i ? a.v_pages : a.k_pages), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            C::INB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kernel = tail_attn_kernel<HD, FP8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kernel, dim3(std::min(C::kPerSm * sm_count(), kTailMaxCtas)), dim3(kThreads), C::SMEM, st, tm[0], tm[1], a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_tail_attn(const GroupedAttnArgs& a, int kv_dtype, int hd, cudaStream_t st) {
  auto go = [&](auto fp8) {
    constexpr bool F = decltype(fp8)::value;
    return hd == 64 ? launch<64, F>(a, st) : hd == 128 ? launch<128, F>(a, st) : launch<256, F>(a, st);
  };
  return kv_dtype == TP_BF16 ? go(std::false_type{}) : go(std::true_type{});
}

}  // namespace tpx
