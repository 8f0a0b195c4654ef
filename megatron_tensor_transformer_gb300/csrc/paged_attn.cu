// Decode attention of one new token per request over a paged key-value cache.
//
// Per request m and q head h of kv head g, over the positions j it attends to (its length, or the
// window at its end):
//   s_j = scale q . k_j,   o = sum_j exp(s_j - max) v_j / sum_j exp(s_j - max),   lse = max + ln sum
// in one pass: the running maximum and sum of each row are kept in fp32, and what was summed under a
// smaller maximum is scaled down when it grows (scores are held times log2 e, for ex2).
//
// HBM-bound: the cache is read once, 4 flops per q head and element.  One persistent CTA per SM; the
// work is a list of units (request, kv head, chunk of P positions) split evenly over the CTAs in
// order, so that one long request and many short ones load all SMs alike.  A producer warp keeps a
// ring of stages (k and v of a chunk) full: lane i looks up the page of box i and issues its TMA copy
// (16 to P positions by 128 bytes, 128-byte swizzle), so a chunk of eight pages costs one pass over the
// warp.  Each consumer warp takes 16 positions of every chunk, always of one page: S = Q K^T and
// P V on mma.sync with the kv head's q heads as the 16 MMA rows (tcgen05 would need 128 rows of
// them), so every byte of the cache is read from shared memory once for all of them.
//   bf16 pages: P enters the product as the sum of two bf16 (its rounding and the rest), so P's
//     rounding does not show beside the output's own; the tensor cores have the time.
//   e4m3 pages: the codes are exact in fp16, so the product runs in fp16, on P rounded to fp16 and q
//     divided by a power of two per head that brings its largest value below 2; the heads' scales go to
//     the scores and to the output.
// Where a (request, kv head) ends inside a CTA's run its warps' states are joined through the stage it
// ended in.  One that is split over CTAs leaves a piece per CTA (sum of p v, max, sum) and the CTA that
// counts in last joins the pieces in order.  Every sum's order follows from the lengths and the SM
// count: runs repeat bit for bit.
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

__host__ __device__ constexpr int chunk_positions(int hd) { return hd == 256 ? 64 : 128; }

template <int HD, bool FP8>
struct PCfg {
  static constexpr int P = chunk_positions(HD);
  static constexpr int CW = P / 16;  // consumer warps
  static constexpr int NT = CW * 32;
  static constexpr int ROWB = HD * (FP8 ? 1 : 2);            // bytes of a position
  static constexpr int INB = ROWB < 128 ? ROWB : 128;        // bytes of a box row
  static constexpr int NIB = ROWB / INB;                     // boxes side by side
  static constexpr int KVB = P * ROWB, STAGE = 2 * KVB;
  static constexpr int NS = (192 * 1024) / STAGE;
  static constexpr int QSTR = HD * 2 + 16;                   // padded q row (bytes)
  static constexpr bool QREG = HD <= 128;                    // q fragments stay in registers
  // the warps' states [16][HD] fp32 fill one stage, or two: then half of the warps join the others first
  static constexpr int RW = STAGE / (16 * HD * 4);           // states a stage holds
  static_assert(RW == CW || RW * 2 == CW, "a stage holds all the warps' states or half of them");
  static constexpr size_t kRing = (size_t)NS * STAGE, kQ = 16 * QSTR;
  static constexpr size_t kML = 2 * 2 * CW * 16 * 4;         // maxima and sums, two buffers
  static constexpr size_t SMEM = 1024 + kRing + kQ + kML + 16 * 4 + (2 * NS + 1) * 8 + NS * 4;
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// two e4m3 codes (low 16 bits) -> two fp16, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xffffu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// what a sum taken under maximum m counts under the maximum mx (0 where nothing was summed)
__device__ __forceinline__ float weight(float m, float mx) { return m == -INFINITY ? 0.f : ex2(m - mx); }

// Byte offset of 16-byte piece j of position r in a chunk: boxes of [P][INB bytes] side by side,
// swizzled as TMA writes them.
template <class C>
__device__ __forceinline__ uint32_t piece_off(int r, int j) {
  constexpr int PB = C::INB / 16;
  const int sw = C::INB == 128 ? (r & 7) : ((r >> 1) & 3);
  return (uint32_t)((j / PB) * (C::P * C::INB) + r * C::INB + (((j % PB) ^ sw) << 4));
}

// The positions [lo, n) a request attends to, in chunks [c0, c1); c0 == c1 if there are none.
struct Span {
  int lo, n, c0, c1;
};
template <int P>
__device__ __forceinline__ Span span_of(const PagedAttnArgs& a, int m) {
  Span s{0, a.lens[m], 0, 0};
  if (s.n < 1 || (long long)s.n > ((long long)a.max_pages << a.page_shift)) return s;
  if (a.window > 0) s.lo = max(0, s.n - a.window);
  s.c0 = s.lo / P;
  s.c1 = (s.n - 1) / P + 1;
  return s;
}

struct Cursor {
  int m, gg, c;
  Span s;
};
template <int P>
__device__ __forceinline__ void advance(const PagedAttnArgs& a, Cursor& cu) {  // only when there is a next unit
  if (++cu.c < cu.s.c1) return;
  if (++cu.gg == a.n_kv) {
    cu.gg = 0;
    do {
      ++cu.m;
      cu.s = span_of<P>(a, cu.m);
    } while (cu.s.c0 == cu.s.c1 && cu.m + 1 < a.M);
  }
  cu.c = cu.s.c0;
}

// CTA i of nct (at most U) takes units [U i / nct, U (i + 1) / nct); owner(u) is the CTA of unit u.
__device__ __forceinline__ long long split_at(long long U, int nct, int i) { return U * i / nct; }
__device__ __forceinline__ int owner(long long U, int nct, long long u) {
  return (int)(((u + 1) * nct + U - 1) / U) - 1;
}

// grid: one CTA per SM; block: CW consumer warps, then the producer warp.
template <int HD, bool FP8>
__global__ void __launch_bounds__(PCfg<HD, FP8>::NT + 32, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ PagedAttnArgs a) {
  using C = PCfg<HD, FP8>;
  extern __shared__ __align__(1024) uint8_t sm_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = ring + C::kRing;                                        // [16][QSTR], rows >= G zero
  float* mlw = reinterpret_cast<float*>(sQ + C::kQ);                    // [2][2][CW][16] maxima, sums
  float* q_pow = mlw + 4 * C::CW * 16;                                  // [16] the rows' power of two (e4m3)
  uint64_t* bars = reinterpret_cast<uint64_t*>(q_pow + 16);             // full[NS], empty[NS], consumers
  uint32_t* loaded = reinterpret_cast<uint32_t*>(bars + 2 * C::NS + 1); // [NS] the boxes a stage holds, by bit
  __shared__ long long s_part[C::CW + 1], s_off;
  __shared__ int s_m, s_last[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const uint32_t full0 = tc::smem_u32(bars), empty0 = full0 + 8 * C::NS, cbar = empty0 + 8 * C::NS;
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      tc::mbar_init(full0 + 8 * i, 1);
      tc::mbar_init(empty0 + 8 * i, C::CW);
    }
    tc::mbar_init(cbar, C::CW);
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  const int G = a.n_q / a.n_kv, nkvs = a.n_kv / a.t;

  // rows without positions
  for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
    const Span s = span_of<C::P>(a, m);
    if (s.c0 != s.c1) continue;
    uint4* o = reinterpret_cast<uint4*>(a.o + (size_t)m * a.n_q * HD);
    for (int i = tid; i < a.n_q * HD / 8; i += C::NT + 32) o[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = tid; i < a.n_q; i += C::NT + 32) a.lse[(size_t)m * a.n_q + i] = -INFINITY;
  }

  // the units: a sum over the requests, a contiguous run of them per thread
  const int per = (a.M + C::NT + 31) / (C::NT + 32), r0 = min(a.M, tid * per), r1 = min(a.M, r0 + per);
  long long here = 0;
  for (int m = r0; m < r1; ++m) {
    const Span s = span_of<C::P>(a, m);
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
  for (int w = 0; w <= C::CW; ++w) {
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
      const Span s = span_of<C::P>(a, m);
      const long long n = (long long)(s.c1 - s.c0) * a.n_kv;
      if (off < n) break;
      off -= n;
    }
    s_m = m;
    s_off = off;
  }
  __syncthreads();
  const int nu = (int)(u1 - u0);
  Cursor cu;
  cu.m = s_m;
  cu.s = span_of<C::P>(a, cu.m);
  cu.gg = (int)(s_off / (cu.s.c1 - cu.s.c0));
  cu.c = cu.s.c0 + (int)(s_off % (cu.s.c1 - cu.s.c0));

  const int box_rows = min(1 << a.page_shift, C::P);
  if (warp == C::CW) {  // producer
    const int nbp = C::P / box_rows;  // boxes along the positions: lane = (kv * NIB + side) * nbp + box
    const int box = lane % nbp, side = lane / nbp % C::NIB, kv = lane / (nbp * C::NIB);
    const uint64_t pol = tc::l2_evict_first();  // the cache streams through once
    auto page_of = [&](const Cursor& x) {  // the page id of this lane's box, -1: nothing to load
      const int p = x.c * C::P + box * box_rows;
      if (kv > 1 || p >= x.s.n || p + box_rows <= x.s.lo) return -1;
      return a.table[(size_t)x.m * a.table_stride + (p >> a.page_shift)];
    };
    int id = page_of(cu);
    for (int k = 0; k < nu; ++k) {
      Cursor nx = cu;
      if (k + 1 < nu) advance<C::P>(a, nx);
      const int next_id = k + 1 < nu ? page_of(nx) : -1;  // in flight while the stage is waited for
      const int st = k % C::NS;
      if (k >= C::NS && !tc::mbar_wait(empty0 + 8 * st, ((k / C::NS) - 1) & 1)) {
        if (lane == 0) atomicExch(a.err, 44u);
        return;
      }
      const bool load = id >= 0 && id < a.n_pages;
      const unsigned boxes = __ballot_sync(kFull, load);
      const uint32_t fb = full0 + 8 * st;
      if (lane == 0) {
        loaded[st] = boxes & ((1u << nbp) - 1);
        tc::mbar_arrive_expect_tx(fb, __popc(boxes) * box_rows * C::INB);
      }
      __syncwarp();
      if (load) {
        const int p = cu.c * C::P + box * box_rows;
        const int row = ((((cu.gg / nkvs) * a.n_pages + id) * nkvs + cu.gg % nkvs) << a.page_shift) +
                        (p & ((1 << a.page_shift) - 1));
        const uint32_t dst = tc::smem_u32(ring + (size_t)st * C::STAGE) + kv * C::KVB + side * (C::P * C::INB) +
                             box * box_rows * C::INB;
        tc::tma_load_2d_hint(dst, kv ? &tmV : &tmK, side * (C::INB / (FP8 ? 1 : 2)), row, fb, pol);
      }
      cu = nx;
      id = next_id;
    }
    return;
  }

  // consumers: warp w takes positions 16w .. 16w+15 of every chunk
  const int gq = lane >> 2, qq = lane & 3, w0 = 16 * warp;
  const uint32_t q_base = tc::smem_u32(sQ);
  uint32_t cph = 0;
  auto csync = [&]() -> bool {  // the consumer warps meet (bounded wait)
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(cbar);
    const bool ok = tc::mbar_wait(cbar, cph);
    cph ^= 1u;
    __syncwarp();
    if (!ok && lane == 0) atomicExch(a.err, 46u);
    return ok;
  };
  // q of a (request, kv head): G heads as 16 rows, QV 16-byte pieces a thread
  constexpr int RP = HD / 8;  // pieces of a row: 8, 16 or 32 neighbouring lanes
  constexpr int QV = (16 * RP + C::NT - 1) / C::NT;
  uint4 qn[QV];
  auto load_q = [&](const Cursor& x) {
    const __nv_bfloat16* qp = a.q + ((size_t)x.m * a.n_q + (size_t)x.gg * G) * HD;
#pragma unroll
    for (int i = 0; i < QV; ++i) {
      const int idx = tid + i * C::NT, r = idx / RP, c8 = idx % RP;
      qn[i] = r < G ? *reinterpret_cast<const uint4*>(qp + (size_t)r * HD + 8 * c8) : make_uint4(0, 0, 0, 0);
    }
  };
  auto store_q = [&]() {
#pragma unroll
    for (int i = 0; i < QV; ++i) {
      const int idx = tid + i * C::NT, r = idx / RP, c8 = idx % RP;
      if (FP8) {  // fp16 of q / 2^e, e the row's largest exponent
        const uint32_t w[4] = {qn[i].x, qn[i].y, qn[i].z, qn[i].w};
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max((w[j] >> 7) & 0xffu, (w[j] >> 23) & 0xffu));
#pragma unroll
        for (int o = 1; o < RP; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
        // exponent fields: 255 (inf, NaN) divides by 2^127, below 2^-126 by 2^-126, so both factors are normal
        const int e = min(max((int)top, 1), 253) - 127;
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = pack_f16(bf16_lo(w[j]) * inv, bf16_hi(w[j]) * inv);
        if (idx < 16 * RP) {
          *reinterpret_cast<uint4*>(sQ + r * C::QSTR + 16 * c8) = make_uint4(h[0], h[1], h[2], h[3]);
          if (c8 == 0) q_pow[r] = __uint_as_float((uint32_t)(127 + e) << 23);
        }
      } else if (idx < 16 * RP) {
        *reinterpret_cast<uint4*>(sQ + r * C::QSTR + 16 * c8) = qn[i];
      }
    }
  };
  // A fragment of 16 dims of q.  e4m3: the k index runs over the dims in the order in which a thread
  // holds four neighbouring codes (2qq + e is dim 4qq + e, 8 + 2qq + e is dim 4qq + 2 + e).
  auto q_frag = [&](int k, uint32_t (&f)[4]) {
    if (FP8) {
      const uint2 lo = *reinterpret_cast<const uint2*>(sQ + gq * C::QSTR + (16 * k + 4 * qq) * 2);
      const uint2 hi = *reinterpret_cast<const uint2*>(sQ + (gq + 8) * C::QSTR + (16 * k + 4 * qq) * 2);
      f[0] = lo.x;
      f[1] = hi.x;
      f[2] = lo.y;
      f[3] = hi.y;
    } else {
      ldsm_x4(q_base + (lane & 15) * C::QSTR + (16 * k + 8 * (lane >> 4)) * 2, f[0], f[1], f[2], f[3]);
    }
  };
  uint32_t qf[C::QREG ? HD / 16 : 1][4];
  float sc0 = 0.f, sc1 = 0.f;  // score factors of rows gq and gq + 8, log2 e included
  auto take_q = [&](const Cursor& x) {
    sc0 = sc1 = a.scale * kLog2e;
    if (FP8) {
      const float ks = a.k_scale ? a.k_scale[x.gg] : 1.0f;
      sc0 *= ks * q_pow[gq];
      sc1 *= ks * q_pow[gq + 8];
    }
    if (C::QREG)
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) q_frag(k, qf[k]);
  };
  load_q(cu);
  store_q();
  if (!csync()) return;
  take_q(cu);

  float O[HD / 8][4];
#pragma unroll
  for (int t8 = 0; t8 < HD / 8; ++t8) O[t8][0] = O[t8][1] = O[t8][2] = O[t8][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows gq and gq + 8
  int c_seg = cu.c;                                          // first chunk of the current piece
  // a split (request, kv head) can only be this CTA's first or last
  int np_mine = 0, pm[2], pgg[2], pa[2], pb[2];
  bool pst[2];  // the first of its CTAs starts with it
  bool first_seg = true;
  int sb = 0;  // which max / sum buffer the next piece end uses
  float* part = reinterpret_cast<float*>(a.ws + kPagedMaxCtas);
  const int per_piece = (G * (HD + 2) + 3) / 4 * 4;
  for (int k = 0; k < nu; ++k) {
    const int st = k % C::NS;
    if (!tc::mbar_wait(full0 + 8 * st, (k / C::NS) & 1)) {
      if (lane == 0) atomicExch(a.err, 45u);
      return;
    }
    const bool last = k + 1 == nu;
    const bool seg_end = last || cu.c + 1 == cu.s.c1;
    uint8_t* stage = ring + (size_t)st * C::STAGE;
    // this warp's positions that count: [a0, a1) of its 16
    const int p0 = cu.c * C::P + w0, a0 = max(0, cu.s.lo - p0), a1 = min(16, cu.s.n - p0);
    const bool work = a0 < a1 && (loaded[st] >> (w0 / box_rows) & 1);
    Cursor nx = cu;
    if (!last) advance<C::P>(a, nx);
    if (seg_end && !last) load_q(nx);  // in flight while this chunk is computed
    if (work) {
      const uint32_t kb = tc::smem_u32(stage), vb = kb + C::KVB;
      if (a1 - a0 < 16) {  // rows that do not count may hold anything (NaN too): P V must see 0
        for (int i = lane; i < 16 * (C::ROWB / 16); i += 32) {
          const int r = i / (C::ROWB / 16), j = i % (C::ROWB / 16);
          if (r < a0 || r >= a1)
            *reinterpret_cast<uint4*>(stage + C::KVB + piece_off<C>(w0 + r, j)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // ordered before the producer's next copy into this stage
        __syncwarp();
      }
      // S = Q K^T over the 16 positions: two n-tiles of 8
      float S[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.f;
      if (FP8) {
#pragma unroll
        for (int k2 = 0; k2 < HD / 32; ++k2) {  // 32 dims: matrices (positions +0, +8) x (dims +0, +16)
          uint32_t b[4], f0[4], f1[4];
          ldsm_x4(kb + piece_off<C>(w0 + (lane & 7) + 8 * ((lane >> 3) & 1), 2 * k2 + (lane >> 4)), b[0], b[1], b[2],
                  b[3]);
          if (!C::QREG) {
            q_frag(2 * k2, f0);
            q_frag(2 * k2 + 1, f1);
          }
          const uint32_t(&x0)[4] = C::QREG ? qf[C::QREG ? 2 * k2 : 0] : f0;
          const uint32_t(&x1)[4] = C::QREG ? qf[C::QREG ? 2 * k2 + 1 : 0] : f1;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma_f16_16816(S[j], x0[0], x0[1], x0[2], x0[3], e4m3x2_to_f16x2(b[j]), e4m3x2_to_f16x2(b[j] >> 16));
            mma_f16_16816(S[j], x1[0], x1[1], x1[2], x1[3], e4m3x2_to_f16x2(b[2 + j]),
                          e4m3x2_to_f16x2(b[2 + j] >> 16));
          }
        }
      } else {
#pragma unroll
        for (int k2 = 0; k2 < HD / 32; ++k2) {
          uint32_t f0[4], f1[4];
          if (!C::QREG) {
            q_frag(2 * k2, f0);
            q_frag(2 * k2 + 1, f1);
          }
          const uint32_t(&x0)[4] = C::QREG ? qf[C::QREG ? 2 * k2 : 0] : f0;
          const uint32_t(&x1)[4] = C::QREG ? qf[C::QREG ? 2 * k2 + 1 : 0] : f1;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t b0, b1, b2, b3;  // positions w0 + 8j + (0..7) x dims 32 k2 + 0/8/16/24
            ldsm_x4(kb + piece_off<C>(w0 + 8 * j + (lane & 7), 4 * k2 + (lane >> 3)), b0, b1, b2, b3);
            mma_bf16_16816(S[j], x0[0], x0[1], x0[2], x0[3], b0, b1);
            mma_bf16_16816(S[j], x1[0], x1[1], x1[2], x1[3], b2, b3);
          }
        }
      }
      // scale, mask, online softmax; a row whose scores are all -inf stays at weight 0
      float mx0 = m0, mx1 = m1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * j + 2 * qq + (i & 1);
          S[j][i] = r >= a0 && r < a1 ? S[j][i] * (i < 2 ? sc0 : sc1) : -INFINITY;
        }
        mx0 = fmaxf(mx0, fmaxf(S[j][0], S[j][1]));
        mx1 = fmaxf(mx1, fmaxf(S[j][2], S[j][3]));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, o));
      }
      if (__any_sync(kFull, mx0 != m0 || mx1 != m1)) {
        const float al0 = weight(m0, mx0), al1 = weight(m1, mx1);
        l0 *= al0;
        l1 *= al1;
#pragma unroll
        for (int t8 = 0; t8 < HD / 8; ++t8) {
          O[t8][0] *= al0;
          O[t8][1] *= al0;
          O[t8][2] *= al1;
          O[t8][3] *= al1;
        }
        m0 = mx0;
        m1 = mx1;
      }
      const float b0x = m0 == -INFINITY ? 0.f : m0, b1x = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        S[j][0] = ex2(S[j][0] - b0x);
        S[j][1] = ex2(S[j][1] - b0x);
        S[j][2] = ex2(S[j][2] - b1x);
        S[j][3] = ex2(S[j][3] - b1x);
      }
      l0 += (S[0][0] + S[0][1]) + (S[1][0] + S[1][1]);  // this lane's share; quad-summed at the end
      l1 += (S[0][2] + S[0][3]) + (S[1][2] + S[1][3]);
      // O += P V: the S fragments are the A fragment of the 16-position k-step
      const int r = w0 + (lane & 7) + 8 * ((lane >> 3) & 1);
      if (FP8) {
        const uint32_t p0f = pack_f16(S[0][0], S[0][1]), p1f = pack_f16(S[0][2], S[0][3]);
        const uint32_t p2f = pack_f16(S[1][0], S[1][1]), p3f = pack_f16(S[1][2], S[1][3]);
#pragma unroll
        for (int t32 = 0; t32 < HD / 32; ++t32) {
          uint32_t v[4];  // (positions +0 / +8) x (dims 32 t32 + 0 / + 16), transposed as pairs of codes
          ldsm_x4_t(vb + piece_off<C>(r, 2 * t32 + (lane >> 4)), v[0], v[1], v[2], v[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // bytes: pos 2qq dims 2gq, 2gq+1, pos 2qq+1 the same
            const uint32_t x = __byte_perm(v[2 * h], 0, 0x3120), y = __byte_perm(v[2 * h + 1], 0, 0x3120);
            float(&even)[4] = O[4 * t32 + 2 * h];
            float(&odd)[4] = O[4 * t32 + 2 * h + 1];
            mma_f16_16816(even, p0f, p1f, p2f, p3f, e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y));
            mma_f16_16816(odd, p0f, p1f, p2f, p3f, e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(y >> 16));
          }
        }
      } else {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = S[i >> 1][2 * (i & 1)], y = S[i >> 1][2 * (i & 1) + 1];
          hi[i] = pack_bf16(x, y);
          lo[i] = pack_bf16(x - bf16_lo(hi[i]), y - bf16_hi(hi[i]));
        }
#pragma unroll
        for (int t16 = 0; t16 < HD / 16; ++t16) {
          uint32_t b0, b1, b2, b3;  // (positions +0 / +8) x (dims 16 t16 + 0 / + 8), transposed
          ldsm_x4_t(vb + piece_off<C>(r, 2 * t16 + (lane >> 4)), b0, b1, b2, b3);
          mma_bf16_16816(O[2 * t16], hi[0], hi[1], hi[2], hi[3], b0, b1);
          mma_bf16_16816(O[2 * t16 + 1], hi[0], hi[1], hi[2], hi[3], b2, b3);
          mma_bf16_16816(O[2 * t16], lo[0], lo[1], lo[2], lo[3], b0, b1);
          mma_bf16_16816(O[2 * t16 + 1], lo[0], lo[1], lo[2], lo[3], b2, b3);
        }
      }
    }
    if (seg_end) {
      // The piece of (m, gg) in this CTA ends: the warps' states join through this stage's memory,
      // then the stage goes back to the producer.
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        l0 += __shfl_xor_sync(kFull, l0, o);
        l1 += __shfl_xor_sync(kFull, l1, o);
      }
      // two buffers: a warp may reach the next piece end while another still reads these
      float* mw = mlw + sb * 2 * C::CW * 16;
      float* lw = mw + C::CW * 16;
      sb ^= 1;
      auto put_ml = [&](int slot) {
        if (qq == 0) {
          mw[slot * 16 + gq] = m0;
          mw[slot * 16 + gq + 8] = m1;
          lw[slot * 16 + gq] = l0;
          lw[slot * 16 + gq + 8] = l1;
        }
      };
      // A state in the stage: row r at r * HD, its 8-float groups permuted by r & 7.  A thread's
      // values are dims 8 t8 + 2qq, + 1 of a bf16 tile and 16 t + 4qq .. + 3 of a pair of e4m3 tiles.
      auto put_O = [&](int slot) {
        float* w = reinterpret_cast<float*>(stage) + (size_t)slot * 16 * HD;
        if (FP8) {
#pragma unroll
          for (int t16 = 0; t16 < HD / 16; ++t16) {
            const int d = (16 * t16 + 4 * qq) ^ ((gq & 7) << 3);
            *reinterpret_cast<float4*>(w + gq * HD + d) =
                make_float4(O[2 * t16][0], O[2 * t16 + 1][0], O[2 * t16][1], O[2 * t16 + 1][1]);
            *reinterpret_cast<float4*>(w + (gq + 8) * HD + d) =
                make_float4(O[2 * t16][2], O[2 * t16 + 1][2], O[2 * t16][3], O[2 * t16 + 1][3]);
          }
        } else {
#pragma unroll
          for (int t8 = 0; t8 < HD / 8; ++t8) {
            const int d = ((8 * t8) ^ ((gq & 7) << 3)) + 2 * qq;
            *reinterpret_cast<float2*>(w + gq * HD + d) = make_float2(O[t8][0], O[t8][1]);
            *reinterpret_cast<float2*>(w + (gq + 8) * HD + d) = make_float2(O[t8][2], O[t8][3]);
          }
        }
      };
      if (!csync()) return;  // every warp is past this chunk's reads of the stage and of sQ
      if (C::RW < C::CW) {   // the upper half of the warps joins the lower half
        if (warp >= C::RW) {
          put_O(warp - C::RW);
          put_ml(warp - C::RW);
        }
        if (!csync()) return;
        if (warp < C::RW) {
          const float* w = reinterpret_cast<const float*>(stage) + (size_t)warp * 16 * HD;
          const float om0 = mw[warp * 16 + gq], om1 = mw[warp * 16 + gq + 8];
          const float ol0 = lw[warp * 16 + gq], ol1 = lw[warp * 16 + gq + 8];
          const float x0 = fmaxf(m0, om0), x1 = fmaxf(m1, om1);
          const float f0 = weight(m0, x0), f1 = weight(m1, x1), g0 = weight(om0, x0), g1 = weight(om1, x1);
          m0 = x0;
          m1 = x1;
          l0 = l0 * f0 + ol0 * g0;
          l1 = l1 * f1 + ol1 * g1;
#pragma unroll
          for (int t16 = 0; t16 < HD / 16; ++t16) {  // e4m3 tiles (bf16 ones fit in one go)
            const int d = (16 * t16 + 4 * qq) ^ ((gq & 7) << 3);
            const float4 y0 = *reinterpret_cast<const float4*>(w + gq * HD + d);
            const float4 y1 = *reinterpret_cast<const float4*>(w + (gq + 8) * HD + d);
            O[2 * t16][0] = O[2 * t16][0] * f0 + y0.x * g0;
            O[2 * t16 + 1][0] = O[2 * t16 + 1][0] * f0 + y0.y * g0;
            O[2 * t16][1] = O[2 * t16][1] * f0 + y0.z * g0;
            O[2 * t16 + 1][1] = O[2 * t16 + 1][1] * f0 + y0.w * g0;
            O[2 * t16][2] = O[2 * t16][2] * f1 + y1.x * g1;
            O[2 * t16 + 1][2] = O[2 * t16 + 1][2] * f1 + y1.y * g1;
            O[2 * t16][3] = O[2 * t16][3] * f1 + y1.z * g1;
            O[2 * t16 + 1][3] = O[2 * t16 + 1][3] * f1 + y1.w * g1;
          }
        }
        __syncwarp();  // a warp reads and then writes its own slot
      }
      if (warp < C::RW) {
        put_O(warp);
        put_ml(warp);
      }
      if (!last) store_q();  // the next piece's q (sQ is free: every warp is past the first csync)
      if (!csync()) return;
      const float* red = reinterpret_cast<const float*>(stage);
      const size_t row = (size_t)cu.m * a.n_q + (size_t)cu.gg * G;  // of o and lse
      const bool whole = c_seg == cu.s.c0 && cu.c + 1 == cu.s.c1;
      const float vs = FP8 && a.v_scale ? a.v_scale[cu.gg] : 1.0f;
      float* piece = part + (size_t)(2 * blockIdx.x + (first_seg ? 0 : 1)) * per_piece;
      for (int e = tid; e < G * HD; e += C::NT) {  // the states under the common maximum, in warp order
        const int hi = e / HD, d = e % HD, ds = d ^ ((hi & 7) << 3);
        float Mx = mw[hi];
#pragma unroll
        for (int w = 1; w < C::RW; ++w) Mx = fmaxf(Mx, mw[w * 16 + hi]);
        float v = 0.f, Lx = 0.f;
#pragma unroll
        for (int w = 0; w < C::RW; ++w) {
          const float f = weight(mw[w * 16 + hi], Mx);
          v += red[((size_t)w * 16 + hi) * HD + ds] * f;
          Lx += lw[w * 16 + hi] * f;
        }
        if (whole) {
          a.o[row * HD + e] = __float2bfloat16_rn(Lx == 0.f ? 0.f : v / Lx * vs);
          if (a.lse && d == 0) a.lse[row + hi] = (Mx + log2f(Lx)) * kLn2;  // -inf + log2(0) where nothing counts
        } else {
          piece[e] = v;
          if (d == 0) {
            piece[G * HD + hi] = Mx;
            piece[G * HD + G + hi] = Lx;
          }
        }
      }
      if (!whole) {
        const long long ub = u0 + k - (cu.c - cu.s.c0);  // the unit of chunk c0 of (m, gg)
        const int i = np_mine++;
        pm[i & 1] = cu.m;
        pgg[i & 1] = cu.gg;
        pa[i & 1] = owner(U, nct, ub);
        pst[i & 1] = split_at(U, nct, pa[i & 1]) == ub;
        pb[i & 1] = owner(U, nct, ub + (cu.s.c1 - cu.s.c0) - 1);
      }
      first_seg = false;
      // The stage returns to the producer once every warp has arrived below, each after its
      // own reads of it; the generic writes to it are ordered before the next copy.
      fence_proxy_async_smem();
      if (!last) take_q(nx);
#pragma unroll
      for (int t8 = 0; t8 < HD / 8; ++t8) O[t8][0] = O[t8][1] = O[t8][2] = O[t8][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
      c_seg = nx.c;
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(empty0 + 8 * st);  // the stage goes back to the producer
    cu = nx;
  }

  // Split (request, kv head)s: count this CTA's pieces in; the CTA that brings the last one joins
  // them all, in order, and leaves the counter at zero.
  if (np_mine == 0) return;
  __threadfence();
  if (!csync()) return;
  if (tid == 0) {
    for (int i = 0; i < np_mine; ++i) {
      const bool is_last = atomicAdd(a.ws + pa[i], 1u) == (unsigned)(pb[i] - pa[i]);
      if (is_last) a.ws[pa[i]] = 0u;
      s_last[i] = is_last;
    }
    __threadfence();
  }
  if (!csync()) return;
  for (int i = 0; i < np_mine; ++i) {
    if (!s_last[i]) continue;
    const size_t row = (size_t)pm[i] * a.n_q + (size_t)pgg[i] * G;
    const float vs = FP8 && a.v_scale ? a.v_scale[pgg[i]] : 1.0f;
    // CTA j's piece is its first one (slot 2 j), but that of the CTA the (request, kv head) starts in
    // only if that CTA's run starts with it
    auto piece_of = [&](int j) { return part + (size_t)(2 * j + (j == pa[i] && !pst[i] ? 1 : 0)) * per_piece; };
    for (int e = 4 * tid; e < G * HD; e += 4 * C::NT) {
      const int hi = e / HD;
      float Mx = -INFINITY, Lx = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int j = pa[i]; j <= pb[i]; ++j) Mx = fmaxf(Mx, __ldcg(piece_of(j) + G * HD + hi));
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
      const float r = Lx == 0.f ? 0.f : vs / Lx;
      *reinterpret_cast<uint2*>(a.o + row * HD + e) = make_uint2(pack_bf16(v.x * r, v.y * r), pack_bf16(v.z * r, v.w * r));
      if (a.lse && e % HD == 0) a.lse[row + hi] = (Mx + log2f(Lx)) * kLn2;
    }
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

template <int HD, bool FP8>
cudaError_t launch(const PagedAttnArgs& a, const void* k_pages, const void* v_pages, cudaStream_t st) {
  using C = PCfg<HD, FP8>;
  EncodeTiled enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap tm[2];
  const int page = 1 << a.page_shift;
  for (int i = 0; i < 2; ++i) {  // the pages as rows of positions
    const cuuint64_t dims[2] = {(cuuint64_t)HD, (cuuint64_t)a.t * a.n_pages * (a.n_kv / a.t) * page};
    const cuuint64_t strides[1] = {(cuuint64_t)C::ROWB};
    const cuuint32_t box[2] = {(cuuint32_t)(C::INB / (FP8 ? 1 : 2)), (cuuint32_t)std::min(page, C::P)}, es[2] = {1, 1};
    if (enc(&tm[i], FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(i ? v_pages : k_pages), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            C::INB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kernel = paged_attn_kernel<HD, FP8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sm_count(), kPagedMaxCtas);
  e = launch_dependent(kernel, dim3(grid), dim3(C::NT + 32), C::SMEM, st, tm[0], tm[1], a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t paged_attn_workspace_bytes(int G, int hd) {
  return (kPagedMaxCtas + 2 * kPagedMaxCtas * piece_floats(G, hd)) * 4;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int kv_dtype, int hd, const void* k_pages, const void* v_pages,
                              cudaStream_t st) {
  if (kv_dtype == TP_BF16) {
    if (hd == 64) return launch<64, false>(a, k_pages, v_pages, st);
    if (hd == 128) return launch<128, false>(a, k_pages, v_pages, st);
    return launch<256, false>(a, k_pages, v_pages, st);
  }
  if (hd == 64) return launch<64, true>(a, k_pages, v_pages, st);
  if (hd == 128) return launch<128, true>(a, k_pages, v_pages, st);
  return launch<256, true>(a, k_pages, v_pages, st);
}

}  // namespace tpx
