// Decode attention of requests that share prefixes: what a group of requests has in common is attended to once.
//
// For one (group, kv head) the rows are (request, q head) pairs, R of them, and the keys the P shared positions:
//   S = scale Q K^T,  ref = max S (running),  P = exp(S - ref),  O += P V,  l += sum P
// and a row's parts (its pieces of the shared positions, and its own positions from tail_attn.cu) are joined by
// their references and sums.  4 R P hd flops over 4 P hd bytes: from 285 rows on the tensor cores bound it, below the HBM.
//
// One persistent CTA per SM takes an even share of the (tile of rows, chunk of 128 positions) list.  A tile is 256 rows
// as two blocks of 128 (128 dims and fewer), or 128 rows.  Products on tcgen05, 128 rows by 128 positions:
//   S = Q K^T   both from shared memory, into tensor memory
//   O += P V    P from tensor memory, where its rows' threads wrote it over S; V as TMA brought it, read transposed
// Over bf16 pages P is two bf16, the upper halves of the weights and what these leave (2^-16 of a weight, as in paged
// attention: half as many bits, 2^-8, showed beside the output's own rounding, 2.3e-3 of o against 1.7e-3).  That is half as
// many MMAs again, 48 of 64 cycles a chunk of 256 rows instead of 32.
// A softmax thread has one row: no shuffles, no shared memory; O stays in tensor memory and is scaled only when a
// row's maximum passes its reference by 2^8.  With two blocks the MMAs of one run beside the exponentials of the
// other; with one, S of the next chunk is computed before P V of this one, into the other half of S.
// e4m3 pages are widened to fp16 in shared memory by four warps (exact), and q is fp16 after a power of two per row.
//
// Measured (one launch, cold; of nominal HBM, of the tensor pipe's cycles): 2048 rows by 30000 positions for each of 8 kv heads
// of 128: 243 us, 44% and 70%, 1.04 PFLOP/s of 4 R P hd, 1.55 with the rests' products; 131072 positions of few rows, 94 us,
// 5.7 TB/s; e4m3, 1536 rows in two groups by 15000: 101 us, 43% of the pipe.  A chunk of a full tile takes 4360 cycles, its MMAs
// 70% of them: of 128 rows S, the exponentials and P V follow one another, and two blocks do not quite cover that; tensor memory has
// no room for a third.  A CTA's beginning (cold code, the groups' scan, q, first copies) took 11 us with P as one bf16, and
// takes 2 to 4 more with the longer code.
#include <cuda.h>

#include <algorithm>

#include "paged_attn.cuh"
#include "tc.h"

namespace tpx {

namespace {

constexpr int kPrefixMaxCtas = 160;
constexpr int kMasks = 32;  // ring of the chunks' masks: above the chunks in flight

template <int HD, bool FP8>
struct XCfg {
  static constexpr int T = HD == 256 ? 1 : 2;           // blocks of 128 rows
  static constexpr int ROWS = 128 * T;
  static constexpr int KS = HD == 256 ? 64 : 128;       // positions per stage
  static constexpr int SUB = kP / KS;
  static constexpr int STAGE = KS * HD * 2;             // k or v in 16 bits: [HD / 64][KS][128 bytes]
  static constexpr int ROWB = HD * (FP8 ? 1 : 2);       // a position as TMA brings it
  static constexpr int INB = ROWB < 128 ? ROWB : 128;
  static constexpr int NIB = ROWB / INB;
  static constexpr int RAW = FP8 ? KS * HD : 0;         // a stage of codes
  static constexpr int NR = FP8 ? (HD == 64 ? 8 : 4) : 0;
  static constexpr int NS = FP8 ? (HD == 64 ? 6 : 3) : (HD == 64 ? 10 : 5);
  static constexpr int NT = FP8 ? NR : NS;              // the ring that TMA fills
  static constexpr int QBLOCK = 128 * HD * 2;
  static constexpr int SMEM = T * QBLOCK + NS * STAGE + NR * RAW;
  static constexpr int kThreads = 128 * T + 128 + (FP8 ? 128 : 0);
  static constexpr float kStep = 8.f;                   // ref may be behind the maximum by this, in powers of two
  static constexpr float kPLog = FP8 ? 7.f : 0.f;       // weights are held times 2^this: at most 2^15 in fp16
  // Units of work: a chunk of a full tile, of one with up to 128 rows, and a tile's beginning and end.  e4m3, two groups of 768
  // rows, with (wide, narrow, ends) of (4, 3, 8) 139 us, (3, 3, 8) 144, (4, 4, 8) 144, (4, 2, 8) 160, (4, 3, 4) 141; bf16 +-1.
  static constexpr int OWN = tail_positions(HD, FP8);   // positions of a stage of a request by itself
  static constexpr int kWide = 4, kNarrow = T == 2 ? 3 : 4, kEnds = 8;
};

struct PrefixArgs {
  GroupedAttnArgs a;
  long long* plan;  // units of all groups, CTAs, then each group's first unit
  float4* whole;    // [n_kv][hd / 4][M G] sum p v of tiles that are not split
  float *whole_ref, *whole_l;  // [n_kv][M G]
  float* pieces;    // [2 kPrefixMaxCtas][piece]
  int piece, rows;  // floats of a piece, rows of its arrays
};

// A group's tiles: of R rows, the last one may have fewer.  0 chunks: nothing is shared.
struct Tiles {
  int full, rest, chunks, len;
  int cost_rest;       // units of a chunk of the last tile
  long long per_head;  // units
};
template <class C>
__device__ __noinline__ Tiles tiles_of(const GroupedAttnArgs& a, int g) {
  Tiles t{};
  const int size = a.cu_groups[g + 1] - a.cu_groups[g];
  t.len = shared_len(a, size, a.prefix_lens[g]);
  t.chunks = (t.len + kP - 1) / kP;
  if (t.chunks == 0) return t;
  const int R = size * (a.n_q / a.n_kv);
  t.full = R / C::ROWS;
  t.rest = R % C::ROWS;
  t.cost_rest = t.rest > 128 ? C::kWide : C::kNarrow;
  t.per_head = (long long)t.full * (C::kEnds + (C::T == 2 ? C::kWide : C::kNarrow) * (long long)t.chunks) +
               (t.rest ? C::kEnds + t.cost_rest * (long long)t.chunks : 0);
  return t;
}

// Chunks [c0, c1) of rows [r0, r0 + rows) of (group, kv head gg); pieces as for paged attention.  g < 0: no more.
struct __align__(16) Tile {
  int g, m0, gg, r0, rows, c0, c1, len, whole, second, pad[2];
};

__device__ __forceinline__ void tmem_ld32(uint32_t t, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&y)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7]), "r"(y[8]), "r"(y[9]),
      "r"(y[10]), "r"(y[11]), "r"(y[12]), "r"(y[13]), "r"(y[14]), "r"(y[15])
      : "memory");
}
// Waits for the loads; the values pass through it, so that no use of them can move before.
template <int N>
__device__ __forceinline__ void landed(float (&v)[N]) {
  tc::tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
// a b + c of two lanes, each rounded once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
template <bool FP8>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (!FP8) return pack_bf16(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// MMAs and what follows them, from a converged warp: one lane, always the same, issues.  (From code that only this lane runs,
// operands are not uniform to the compiler, and moving them took 100 cycles an MMA.)
__device__ __forceinline__ void warp_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void warp_mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void warp_commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(kFull, v, 0); }

// 16-bit operands (bf16, or fp16 with FP8 pages), fp32 sums
template <bool FP8>
__host__ __device__ constexpr uint32_t idesc16(int M, int N) {
  return (1u << 4) | (FP8 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kBTransposed = 1u << 16;  // B is rows of k

// grid: one CTA per SM
template <int HD, bool FP8>
__global__ void __launch_bounds__(XCfg<HD, FP8>::kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ PrefixArgs pa) {
  using C = XCfg<HD, FP8>;
  const GroupedAttnArgs& a = pa.a;
  constexpr int kSoftWarps = 4 * C::T, kProducer = kSoftWarps, kMma = kProducer + 1, kItems = kProducer + 2,
                kWarps = C::kThreads / 32, kWiden = kProducer + 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;                          // [T][HD / 64][128][128 bytes], swizzled
  uint8_t* ring = smem + C::T * C::QBLOCK;     // [NS] stages
  uint8_t* raw = ring + C::NS * C::STAGE;      // [NR] stages of codes
  __shared__ Tile s_tile[4];
  __shared__ __align__(8) uint64_t full[C::NS], empty[C::NS], rfull[C::NR + 1], rempty[C::NR + 1], q_full[2],
      s_full[3], p_full[3], pv_done, o_full[2], i_full[4], i_empty[4], mma_done;
  __shared__ long long s_part[kWarps], s_base;  // s_base: units before group s_g, which holds the CTA's first one
  __shared__ uint32_t loaded[kMasks];           // 16-position groups of a chunk that were loaded, by bit
  __shared__ uint32_t s_tmem;
  __shared__ int s_g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  auto B = [](const uint64_t& b) { return tc::smem_u32(&b); };
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      tc::mbar_init(B(full[i]), FP8 ? 4 : 1);
      tc::mbar_init(B(empty[i]), 1);
    }
    for (int i = 0; i < C::NR; ++i) {
      tc::mbar_init(B(rfull[i]), 1);
      tc::mbar_init(B(rempty[i]), 4);
    }
    tc::mbar_init(B(pv_done), 1);
    tc::mbar_init(B(mma_done), 1);
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(B(s_full[i]), 2);  // the MMAs' commit, and the issuing thread's own arrival
      tc::mbar_init(B(p_full[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(B(q_full[i]), 4);
      tc::mbar_init(B(o_full[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(B(i_full[i]), 1);
      tc::mbar_init(B(i_empty[i]), kSoftWarps + 2 + (FP8 ? 4 : 0));
    }
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  if (warp == kMma) tc::tmem_alloc(tc::smem_u32(&s_tmem), 512);
  tc::griddep_launch_dependents();
  const int G = a.n_q / a.n_kv, nkvs = a.n_kv / a.t;

  // The units: a sum over the groups, a contiguous run of them per thread.
  const bool ok = __syncthreads_and(groups_in_order(a, tid, C::kThreads));
  const int ng = ok ? a.n_groups : 0;
  const int per = (ng + C::kThreads - 1) / C::kThreads, g0 = min(ng, tid * per), g1 = min(ng, g0 + per);
  long long here = 0;
  for (int g = g0; g < g1; ++g) here += tiles_of<C>(a, g).per_head * a.n_kv;
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
  const int nct = (int)min((long long)gridDim.x, U / C::kWide);
  const long long u0 = nct == 0 ? 0 : quot_call(U * min((int)blockIdx.x, nct), nct),
                  u1 = nct == 0 ? 0 : quot_call(U * min((int)blockIdx.x + 1, nct), nct);
  if (blockIdx.x == 0) {  // for the join
    if (tid == 0) {
      pa.plan[0] = U;
      pa.plan[1] = nct;
    }
    long long at = base;
    for (int g = g0; g < g1; ++g) {
      pa.plan[2 + g] = at;
      at += tiles_of<C>(a, g).per_head * a.n_kv;
    }
  }
  if (u0 < u1 && u0 >= base && u0 < base + here) {  // this thread's groups hold unit u0
    int g = g0;
    for (;; ++g) {
      const long long n = tiles_of<C>(a, g).per_head * a.n_kv;
      if (u0 < base + n) break;
      base += n;
    }
    s_g = g;
    s_base = base;
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;
  // Columns of S in 64s: of P for 64 positions the first 32 hold the weights in 16 bits, over bf16 pages the last 32 the rest.
  auto S_at = [&](int r) { return tmem + 128 * r; };
  auto O_at = [&](int x) { return tmem + 256 + HD * x; };
  // Item j as a role sees it.
  auto next_item = [&](Waits& wait, int j, bool whole_warp) {
    wait(B(i_full[j & 3]), (j >> 2) & 1);
    const Tile it = s_tile[j & 3];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) tc::mbar_arrive(B(i_empty[j & 3]));
    if (wait.failed) {  // nothing to go by: end
      Tile none = it;
      none.g = -1;
      return none;
    }
    return it;
  };
  // S and P have a barrier each per region and reader, so that every phase is waited for, in order, by one role: 0 the
  // first block, or even chunks of a tile of one; 1 the odd chunks of those; 2 the second block.
  auto wide = [](const Tile& it) { return C::T == 2 && it.rows > 128; };

  if (warp < kSoftWarps) {
    // ---- softmax: thread = row
    Waits wait{a.err, 58u, false};
    const int x = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    int uses[3] = {0, 0, 0}, kc = 0, pv = 0, done = 0;  // S by barrier, chunks, products of narrow items, items
    int j = 0;
    auto next_tile = [&]() {  // the next item that has rows for this block
      for (;; ++j) {
        const Tile it = next_item(wait, j, true);
        if (__any_sync(kFull, it.g < 0)) {
          Tile none = it;
          none.g = -1;
          return none;
        }
        if (x == 0 || wide(it)) {
          ++j;
          return it;
        }
        kc += it.c1 - it.c0;
      }
    };
    // The warp's 32 rows of q to shared memory, neighbouring lanes along a row (a row per thread took 2 us more): nothing
    // reads the block's q any more once its last S is there.  Returns 2^e by which the thread's row was divided.
    auto bring_q = [&](const Tile& it) {
      constexpr int RP = HD / 8, kRows = 32 / RP;  // 16-byte pieces of a row, rows at once
      const int r = x * 128 + row, R = it.r0 + min(r, it.rows - 1), m = R / G;
      const int at = (it.m0 + m) * a.n_q + it.gg * G + (R - m * G);  // the thread's row of q
      const int c8 = lane % RP, sub = lane / RP;
      float pow = 1.f;
#pragma unroll 2
      for (int i = 0; i < 32; i += kRows) {
        const int l = i + sub, rr = (row & ~31) + l;  // the lane whose row it is, in the block
        const bool there = x * 128 + rr < it.rows;
        const __nv_bfloat16* src = a.q + (size_t)__shfl_sync(kFull, at, l) * HD + 8 * c8;
        uint8_t* dst = sQ + x * C::QBLOCK + (c8 >> 3) * 16384 + rr * 128 + (((c8 & 7) ^ (rr & 7)) << 4);
        if (!FP8) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
                       : "memory");
          continue;
        }
        const uint4 v = there ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
        int e;
        *reinterpret_cast<uint4*>(dst) = q_as_fp16<RP>(v, e);
        const int mine = __shfl_sync(kFull, e, lane % kRows * RP);
        if (lane / kRows * kRows == i) pow = __uint_as_float((uint32_t)mine << 23);
      }
      if (!FP8) asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(B(q_full[x]));
      return pow;
    };
    Tile it = next_tile();
    float pow = it.g >= 0 ? bring_q(it) : 1.f;
    while (it.g >= 0) {
      const int n = it.c1 - it.c0;
      const bool w2 = wide(it);
      float sc = a.scale * kLog2e * (FP8 && a.k_scale ? a.k_scale[it.gg] : 1.0f) * pow, sub = kNoRef, l = 0.f;
      const bool flip = sc < 0.f;
      bool live = false;
      for (int i = 0; i < n; ++i) {
        const int region = w2 ? x : i & 1, b = w2 ? 2 * x : i & 1;
        wait(B(s_full[b]), (b == 0 ? uses[0]++ : b == 1 ? uses[1]++ : uses[2]++) & 1);
        __syncwarp();
        tc::tc_fence_after();
        const uint32_t sA = S_at(region) + lanes;
        const uint32_t groups = loaded[(kc + i) % kMasks];
        // The row is read twice, 64 positions at a time in loops: a row in registers takes no fewer cycles, and code
        // that is long costs where a CTA runs it once or twice (20 cycles an instruction until it is in the cache).
        float top = flip ? INFINITY : -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          float s[64];
          tmem_ld32(sA + c, s);
          tmem_ld32(sA + c + 32, s + 32);
          landed(s);
          if (groups != 0xffu) {
#pragma unroll
            for (int q = 0; q < 64; ++q) s[q] = groups >> (c / 16 + q / 16) & 1 ? s[q] : flip ? INFINITY : -INFINITY;
          }
          if (!flip) {
            float t4[4] = {top, s[61], s[62], s[63]};
#pragma unroll
            for (int q = 0; q < 60; q += 8) {
#pragma unroll
              for (int r = 0; r < 4; ++r) t4[r] = fmaxf(t4[r], q + 4 + r < 61 ? fmaxf(s[q + r], s[q + 4 + r]) : s[q + r]);
            }
            top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          } else {
#pragma unroll
            for (int q = 0; q < 64; ++q) top = fminf(top, s[q]);
          }
        }
        top = __fmul_rn(top, sc);
        const bool raise = top > sub + (C::kStep + C::kPLog);
        if (__any_sync(kFull, raise)) {  // a new reference: the maximum so far
          const float to = raise ? fmaxf(sub, top - C::kPLog) : sub, f = ex2(sub - to);  // from kNoRef: of a sum that is 0
          l *= f;
          sub = to;
          if (live) {
            if (!w2) {
              wait(B(pv_done), (pv + i - 1) & 1);
              __syncwarp();
              tc::tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < HD; c += 16) {
              float o[16];
              tc::tmem_ld16(O_at(x) + lanes + c, o);
              landed(o);
              uint32_t y[16];
#pragma unroll
              for (int q = 0; q < 16; ++q) y[q] = __float_as_uint(o[q] * f);
              tmem_st16(O_at(x) + lanes + c, y);
            }
          }
        }
        // s sc - sub, rounded once: what sub's own rounding adds is the same for all of the row's weights under it, and
        // divides out.  Beyond 2^20 it could be large: there the product is rounded by itself.
        const bool far = !(fabsf(sub) < 1048576.f), any_far = __any_sync(kFull, far);
        const float2 sc2 = make_float2(sc, sc), sub2 = make_float2(-sub, -sub);
        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          float s[64];
          tmem_ld32(sA + c, s);
          tmem_ld32(sA + c + 32, s + 32);
          landed(s);
          if (any_far) {
#pragma unroll
            for (int q = 0; q < 64; ++q) s[q] = far ? __fmul_rn(s[q], sc) - sub : fmaf(s[q], sc, -sub);
          } else {
#pragma unroll
            for (int q = 0; q < 64; q += 2) {
              const float2 y = fma2(make_float2(s[q], s[q + 1]), sc2, sub2);
              s[q] = y.x;
              s[q + 1] = y.y;
            }
          }
          if (groups != 0xffu) {
#pragma unroll
            for (int q = 0; q < 64; ++q) s[q] = groups >> (c / 16 + q / 16) & 1 ? s[q] : -INFINITY;
          }
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t p[16], rest[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float2 y = make_float2(ex2(s[32 * part + 2 * q]), ex2(s[32 * part + 2 * q + 1]));
              l2[q & 1] = add2(l2[q & 1], y);
              if (FP8) {
                p[q] = pack16<true>(y.x, y.y);
              } else {  // the upper halves as they are, and what they leave, rounded: 2^-16 of a weight
                p[q] = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
                rest[q] = pack_bf16(y.x - bf16_lo(p[q]), y.y - bf16_hi(p[q]));
              }
            }
            tmem_st16(sA + c + 16 * part, p);  // over columns that have been read
            if (!FP8) tmem_st16(sA + c + 32 + 16 * part, rest);
          }
        }
        l += (l2[0].x + l2[1].x) + (l2[0].y + l2[1].y);  // a chunk by itself: n / 128 + 34 roundings for n positions
        tc::tmem_st_wait();
        live |= groups != 0;
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(B(p_full[b]));
      }
      kc += n;
      if (!w2) pv += n;

      // The next item's q, then the item's end: O to the joining kernel, a float4 of dims after the other with the rows
      // side by side.  (P for the next item is written behind this: until then its P V leaves O alone.)
      const Tile next = next_tile();
      if (next.g >= 0) pow = bring_q(next);
      wait(B(o_full[x]), done++ & 1);
      __syncwarp();
      tc::tc_fence_after();
      const float vs = FP8 && a.v_scale ? a.v_scale[it.gg] : 1.0f;
      const int r = x * 128 + row, RT = a.M * G, R = it.m0 * G + it.r0 + r;
      const bool whole = it.whole, there = r < it.rows;
      float* piece = pa.pieces + (size_t)(2 * blockIdx.x + it.second) * pa.piece;
      float4* dst = whole ? pa.whole + (size_t)it.gg * (HD / 4) * RT + R : reinterpret_cast<float4*>(piece) + r;
      const size_t step = whole ? RT : pa.rows;
      if (live) {
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float o[32];
          tmem_ld32(O_at(x) + lanes + c, o);
          landed(o);
          if (there) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              dst[(c / 4 + q) * step] = make_float4(o[4 * q] * vs, o[4 * q + 1] * vs, o[4 * q + 2] * vs, o[4 * q + 3] * vs);
          }
        }
      }
      if (there) {
        float* refs = whole ? pa.whole_ref + (size_t)it.gg * RT + R : piece + (size_t)pa.rows * HD + r;
        float* sums = whole ? pa.whole_l + (size_t)it.gg * RT + R : piece + (size_t)pa.rows * (HD + 1) + r;
        *refs = sub;
        *sums = l;
      }
      tc::tc_fence_before();
      __syncwarp();
      it = next;
    }
  } else {
    if (warp == kProducer) {
      // ---- k and v in the order in which the MMAs take them: a stage is SUB-th of a chunk's k or v
      Waits wait{a.err, 59u, false};
      const int box_rows = min(1 << a.page_shift, C::KS), nbp = C::KS / box_rows;  // boxes along the positions
      const int box = lane % nbp, side = lane / nbp;
      int cnt = 0, kc = 0;
      struct Rows {  // a chunk's boxes, this lane's of each stage
        int row[C::SUB];
        unsigned boxes[C::SUB];
      };
      uint8_t* dst = FP8 ? raw : ring;
      constexpr int kBytes = FP8 ? C::RAW : C::STAGE;
      uint64_t(&tfull)[FP8 ? C::NR + 1 : C::NS] = *(FP8 ? reinterpret_cast<uint64_t(*)[FP8 ? C::NR + 1 : C::NS]>(&rfull)
                                                        : reinterpret_cast<uint64_t(*)[FP8 ? C::NR + 1 : C::NS]>(&full));
      uint64_t(&tempty)[FP8 ? C::NR + 1 : C::NS] = *(FP8 ? reinterpret_cast<uint64_t(*)[FP8 ? C::NR + 1 : C::NS]>(&rempty)
                                                         : reinterpret_cast<uint64_t(*)[FP8 ? C::NR + 1 : C::NS]>(&empty));
      auto copy = [&](const CUtensorMap& tm, const Rows& r) {
#pragma unroll
        for (int s = 0; s < C::SUB; ++s, ++cnt) {
          const int st = cnt % C::NT;
          if (cnt >= C::NT) wait(B(tempty[st]), (cnt / C::NT - 1) & 1);
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_expect_tx(B(tfull[st]), __popc(r.boxes[s]) * box_rows * C::INB);
          __syncwarp();
          if (r.boxes[s] >> lane & 1)
            tc::tma_load_2d(tc::smem_u32(dst + (size_t)st * kBytes) + (side * C::KS + box * box_rows) * C::INB, &tm,
                            side * (C::INB / (FP8 ? 1 : 2)), r.row[s], B(tfull[st]));
        }
      };
      bool stop = false;
      for (int j = 0; !stop; ++j) {
        const Tile it = next_item(wait, j, true);
        if (__any_sync(kFull, it.g < 0)) break;
        const int pages0 = (it.gg / nkvs) * a.n_pages, gl = it.gg % nkvs;
        // page ids 32 at a time, one per lane, the next 32 on their way; a chunk's pages never straddle two batches
        int at = it.c0 * kP >> a.page_shift;
        auto ids_from = [&](int page) {
          page += lane;
          return ((long long)page << a.page_shift) < it.len ? a.table[(size_t)it.m0 * a.table_stride + page] : -1;
        };
        int ids = ids_from(at), ids_next = ids_from(at + 32);
        auto look_up = [&](int c, Rows& r) {
          if (((c * kP + kP - 1) >> a.page_shift) >= at + 32) {
            at += 32;
            ids = ids_next;
            ids_next = ids_from(at + 32);
          }
          unsigned groups = 0;
#pragma unroll
          for (int s = 0; s < C::SUB; ++s) {
            const int pos = c * kP + s * C::KS + box * box_rows;
            int id = __shfl_sync(kFull, ids, ((pos >> a.page_shift) - at) & 31);
            if (side >= C::NIB || pos >= it.len) id = -1;
            r.row[s] = (((pages0 + id) * nkvs + gl) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
            r.boxes[s] = __ballot_sync(kFull, id >= 0 && id < a.n_pages);
            const unsigned in = __ballot_sync(kFull, lane < C::KS / 16 && (r.boxes[s] >> ((lane * 16 / box_rows) & 31) & 1));
            groups |= in << (s * (C::KS / 16));
          }
          // seen by who waits for the chunk's k
          if (lane == 0) loaded[kc % kMasks] = groups;
          ++kc;
        };
        Rows now, next;
        if (wide(it)) {
          for (int c = it.c0; c < it.c1 && !stop; ++c) {
            look_up(c, now);
            copy(tmK, now);
            copy(tmV, now);
            stop = __any_sync(kFull, wait.failed);
          }
        } else {
          look_up(it.c0, now);
          copy(tmK, now);
          for (int c = it.c0; c < it.c1 && !stop; ++c) {
            if (c + 1 < it.c1) {
              look_up(c + 1, next);
              copy(tmK, next);
            }
            copy(tmV, now);
            now = next;
            stop = __any_sync(kFull, wait.failed);
          }
        }
      }
      const int last = cnt - 1 - lane;  // copies in flight: each stage's last
      if (lane < C::NT && last >= 0) wait_long(B(tfull[last % C::NT]), (last / C::NT) & 1, a.err, 59u);
    } else if (warp == kMma) {
      // ---- one warp issues all MMAs; they run in the order of issue, so a region of S is written anew behind the
      // product that read P from it
      {
        Waits wait_lane{a.err, 55u, false};
        auto wait = [&](uint32_t bar, uint32_t parity) { return !__any_sync(kFull, !wait_lane(bar, parity)); };
        const uint32_t tmem_u = uniform(tmem);
        auto S_at = [&](int r) { return tmem_u + 128 * r; };
        auto O_at = [&](int x) { return tmem_u + 256 + HD * x; };
        constexpr uint32_t idS = idesc16<FP8>(128, C::KS), idO = idesc16<FP8>(128, HD) | kBTransposed;
        const uint32_t qA = uniform(tc::smem_u32(sQ)), rA = uniform(tc::smem_u32(ring));
        int cnt = 0, kc = 0, uses[3] = {0, 0, 0}, done[2] = {0, 0};  // stages, chunks, S by barrier, blocks' items
        auto take = [&](int& st) {
          st = cnt % C::NS;
          const bool there = wait(B(full[st]), (cnt / C::NS) & 1);
          ++cnt;
          return there;
        };
        // The thread has 64 cycles for an MMA: descriptors are a base and steps (addresses do not carry out of their
        // field).  Loops that made each anew took 140.
        auto scores = [&](int x, int region, int st, int sub) {
          uint64_t q0 = smem_desc(qA + x * C::QBLOCK, 16, 1024, 2), k0 = smem_desc(rA + st * C::STAGE, 16, 1024, 2);
          const uint32_t d = S_at(region) + sub * C::KS;
#pragma unroll 1
          for (int i = 0; i < HD / 64; ++i) {  // 64 dims: rows of 128 bytes
#pragma unroll
            for (int k = 0; k < 4; ++k) warp_mma(d, q0 + tc::desc_off(32 * k), k0 + tc::desc_off(32 * k), idS, i + k > 0);
            q0 += tc::desc_off(16384);
            k0 += tc::desc_off(C::KS * 128);
          }
        };
        auto scores_end = [&](int b) {
          warp_commit(B(s_full[b]));
          if (lane == 0) tc::mbar_arrive(B(s_full[b]));  // releases what this thread has seen: the chunk's mask, q's powers
          b == 0 ? ++uses[0] : b == 1 ? ++uses[1] : ++uses[2];
        };
        auto values = [&](int x, int region, int st, int sub, uint32_t groups, bool& live) {
          const uint64_t v0 = smem_desc(rA + st * C::STAGE, C::KS * 128, 1024, 2);
          const uint32_t p = S_at(region) + sub * C::KS, d = O_at(x);
#pragma unroll 1
          for (int i = 0; i < C::KS / 16; i += 4) {  // 64 positions: 64 columns of P
            if (groups == 0xffu) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                warp_mma_tmem_a(d, p + 16 * i + 8 * k, v0 + tc::desc_off(2048) * (i + k), idO, live);
                if (!FP8) warp_mma_tmem_a(d, p + 16 * i + 32 + 8 * k, v0 + tc::desc_off(2048) * (i + k), idO, true);
                live = true;
              }
              continue;
            }
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              if (!(groups >> (sub * (C::KS / 16) + i + k) & 1)) continue;  // what was not loaded may hold anything
              warp_mma_tmem_a(d, p + 16 * i + 8 * k, v0 + tc::desc_off(2048) * (i + k), idO, live);
              if (!FP8) warp_mma_tmem_a(d, p + 16 * i + 32 + 8 * k, v0 + tc::desc_off(2048) * (i + k), idO, true);
              live = true;
            }
          }
        };
        for (int j = 0;; ++j) {
          const Tile it = next_item(wait_lane, j, true);
          if (__any_sync(kFull, it.g < 0)) break;
          if (!wait(B(q_full[0]), done[0] & 1)) break;
          const int n = (int)uniform(it.c1 - it.c0);
          const bool two = uniform(wide(it)) != 0;
          if (two && !wait(B(q_full[1]), done[1] & 1)) break;
          bool live[2] = {false, false};
          int st, sv;
          if (two) {
            if (!take(st)) goto mma_end;
            tc::tc_fence_after();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              scores(x, x, st, 0);
              scores_end(2 * x);
            }
            warp_commit(B(empty[st]));
            for (int i = 0; i < n; ++i) {
              if (!take(sv)) goto mma_end;
              const uint32_t groups = uniform(loaded[(kc + i) % kMasks]);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                if (!wait(B(p_full[2 * x]), (uses[2 * x] - 1) & 1)) goto mma_end;
                tc::tc_fence_after();
                values(x, x, sv, 0, groups, live[x]);
                if (x == 1) warp_commit(B(empty[sv]));
                if (i + 1 < n) {
                  if (x == 0 && !take(st)) goto mma_end;
                  tc::tc_fence_after();
                  scores(x, x, st, 0);
                  scores_end(2 * x);
                  if (x == 1) warp_commit(B(empty[st]));
                } else {
                  warp_commit(B(o_full[x]));
                  ++done[x];
                }
              }
            }
          } else {
            auto next_scores = [&](int i) {
              for (int sub = 0; sub < C::SUB; ++sub) {
                if (!take(st)) return false;
                tc::tc_fence_after();
                scores(0, i & 1, st, sub);
                warp_commit(B(empty[st]));
              }
              scores_end(i & 1);
              return true;
            };
            if (!next_scores(0)) goto mma_end;
            for (int i = 0; i < n; ++i) {
              const int p_use = (i & 1 ? uses[1] : uses[0]) - 1;
              if (i + 1 < n && !next_scores(i + 1)) goto mma_end;
              if (!wait(B(p_full[i & 1]), p_use & 1)) goto mma_end;
              const uint32_t groups = uniform(loaded[(kc + i) % kMasks]);
              for (int sub = 0; sub < C::SUB; ++sub) {
                if (!take(sv)) goto mma_end;
                tc::tc_fence_after();
                values(0, i & 1, sv, sub, groups, live[0]);
                warp_commit(B(empty[sv]));
              }
              warp_commit(B(pv_done));
            }
            warp_commit(B(o_full[0]));
            ++done[0];
          }
          kc += n;
        }
    mma_end:
        warp_commit(B(mma_done));  // the MMAs in flight
        if (lane == 0) wait_long(B(mma_done), 0, a.err, 55u);
      }
      __syncwarp();
    } else if (warp == kItems) {
      // ---- items
      Waits wait{a.err, 56u, false};
      int g = u0 < u1 ? s_g : 0, gg = 0, tile = 0;
      long long at = u0 < u1 ? s_base : u1;  // the first unit of the tile
      Tiles ts{};
      if (u0 < u1) {  // the tile that holds u0
        ts = tiles_of<C>(a, g);
        gg = (int)quot_call(u0 - at, ts.per_head);
        at += (long long)gg * ts.per_head;
        if (ts.full) {
          const long long one = C::kEnds + (C::T == 2 ? C::kWide : C::kNarrow) * (long long)ts.chunks;
          tile = (int)min((long long)ts.full, quot_call(u0 - at, one));
          at += tile * one;
        }
      }
      for (int j = 0;; ++j) {
        Tile it{};
        it.g = -1;
        if (__any_sync(kFull, wait.failed)) at = u1;  // for all lanes
        while (at < u1) {
          const int ntiles = ts.full + (ts.rest > 0), ch = ts.chunks;
          const int cost = tile < ts.full ? (C::T == 2 ? C::kWide : C::kNarrow) : ts.cost_rest;
          const long long units = ch == 0 ? 0 : C::kEnds + cost * (long long)ch;
          if (ch > 0) {
            // chunk i begins at unit at + kEnds + cost i, and is of the CTA that has this unit
            auto chunks_before = [&](long long u) {
              const long long d = u - at - C::kEnds;
              return d <= 0 ? 0 : d >= cost * (long long)ch ? ch : (int)quot_call(d + cost - 1, cost);
            };
            it.c0 = chunks_before(u0);
            it.c1 = chunks_before(u1);
          }
          if (ch > 0 && it.c0 < it.c1) {
            it.g = g;
            it.m0 = a.cu_groups[g];
            it.gg = gg;
            it.r0 = tile * C::ROWS;
            it.rows = tile < ts.full ? C::ROWS : ts.rest;
            it.len = ts.len;
            it.whole = it.c0 == 0 && it.c1 == ch;
            // a piece is the CTA's second where it begins the tile, and the CTA's run begins before
            it.second = it.c0 == 0 && u0 < at;
          }
          at += units;
          if (++tile >= ntiles || ch == 0) {
            tile = 0;
            if (++gg >= a.n_kv || ch == 0) {
              gg = 0;
              if (++g >= ng) at = u1;
              else ts = tiles_of<C>(a, g);
            }
          }
          if (it.g >= 0) break;
        }
        if (j >= 4) wait(B(i_empty[j & 3]), ((j >> 2) - 1) & 1);
        if (lane == 0) {
          s_tile[j & 3] = it;
          tc::mbar_arrive(B(i_full[j & 3]));
        }
        if (it.g < 0) break;
      }
    } else if (FP8 && warp >= kWiden) {
      // ---- codes to fp16, a stage after the other: thread = position (and half of the dims for stages of 64)
      Waits wait{a.err, 57u, false};
      const int wt = tid - kWiden * 32, r = wt % C::KS;
      int cnt = 0;
      for (int j = 0;; ++j) {
        const Tile it = next_item(wait, j, true);
        if (__any_sync(kFull, it.g < 0)) break;
        for (int f = 0; f < 2 * C::SUB * (it.c1 - it.c0); ++f, ++cnt) {
          const int rs = cnt % max(1, C::NR), ws = cnt % C::NS;
          wait(B(rfull[rs]), (cnt / max(1, C::NR)) & 1);
          if (cnt >= C::NS) wait(B(empty[ws]), (cnt / C::NS - 1) & 1);
          if (__any_sync(kFull, wait.failed)) goto widen_end;
          const uint8_t* src = raw + (size_t)rs * C::RAW + r * C::INB;
          uint8_t* dst = ring + (size_t)ws * C::STAGE + r * 128;
          constexpr int kUnits = HD / 16 / (128 / C::KS);  // 16 codes each
#pragma unroll
          for (int i = 0; i < kUnits; ++i) {
            const int u = i + (wt / C::KS) * kUnits, side = u / (C::INB / 16), p = u % (C::INB / 16);
            const int at = C::INB == 128 ? p ^ (r & 7) : p ^ ((r >> 1) & 3);
            const uint4 v = *reinterpret_cast<const uint4*>(src + side * (C::KS * C::INB) + (at << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const __half2 x = e4m3x2_half2((w[q >> 1] >> (16 * (q & 1))) & 0xffffu);
              h[q] = *reinterpret_cast<const uint32_t*>(&x);
            }
            uint8_t* to = dst + (u >> 2) * (C::KS * 128);
            const int p16 = 2 * (u & 3);
            *reinterpret_cast<uint4*>(to + ((p16 ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(to + (((p16 + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(B(full[ws]));
            tc::mbar_arrive(B(rempty[rs]));
          }
        }
      }
  widen_end:;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc::tc_fence_after();
    tc::tmem_relinquish();
    tc::tmem_dealloc(tmem, 512);
  }
}

// The parts of a row in order: the pieces of what its group shares, then of its own positions.  One block per (request,
// kv head), a float4 of a head's dims per thread; kBatch parts are read at once.
template <int HD, bool FP8>
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ PrefixArgs pa) {
  using C = XCfg<HD, FP8>;
  constexpr int SP = C::OWN, kBatch = 4;
  // What the call was given may be read before the call's other kernels have ended, since the first of them began after all
  // work before the call; what they leave, only after.
  const GroupedAttnArgs& a = pa.a;
  const int m = blockIdx.x / a.n_kv, gg = blockIdx.x % a.n_kv, G = a.n_q / a.n_kv, RT = a.M * G;
  const bool ok = __syncthreads_and(groups_in_order(a, threadIdx.x, blockDim.x));
  const Span s = own_span<SP>(a, m, ok);
  int g = ok ? group_of(a, m) : -1, m0 = 0;
  if (g >= 0 && (s.n < 1 || (long long)s.n > ((long long)a.max_pages << a.page_shift) || left_to_group(a, g, s.n) == 0)) g = -1;
  Tiles ts{};
  if (g >= 0) {
    ts = tiles_of<C>(a, g);
    m0 = a.cu_groups[g];
  }
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  // Which CTAs have parts: of the request's own run, and of the one or two tiles that its rows lie in.  Divisions of 64
  // bits are long, so one warp makes them, a lane each.
  __shared__ int s_cta[3][2], s_second[3];
  const int R0 = (m - m0) * G, tile0 = R0 / C::ROWS;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, what = lane >> 1, tile = tile0 + what - 1;
    long long U = 0, at = 0, u = -1;  // units and CTAs of its list, its first unit, the unit asked for
    int nct = 1;
    if (what == 0) {
      const int ch = s.c1 - s.c0;
      U = a.own_plan[0];
      nct = (int)a.own_plan[1];
      at = a.own_plan[2 + m] + (long long)gg * (kTailEnds + ch);
      if (ch > 0) u = at + kTailEnds + (lane & 1) * (ch - 1);
    } else if (what < 3 && g >= 0 && tile < ts.full + (ts.rest > 0)) {
      const int cost_full = C::T == 2 ? C::kWide : C::kNarrow, cost = tile < ts.full ? cost_full : ts.cost_rest;
      U = pa.plan[0];
      nct = (int)pa.plan[1];
      at = pa.plan[2 + g] + gg * ts.per_head + tile * (C::kEnds + cost_full * (long long)ts.chunks);
      u = at + C::kEnds + (lane & 1) * (cost * (long long)(ts.chunks - 1));
    }
    const int cta = u >= 0 ? owner(U, nct, u) : -(lane & 1);  // none: 0 .. -1
    const bool second = u >= 0 && split_at(U, nct, cta) < at;
    if (lane < 6) {
      s_cta[what][lane & 1] = cta;
      if (!(lane & 1)) s_second[what] = second;
    }
  }
  __syncthreads();
  const int own_a = s_cta[0][0], n_own = s_cta[0][1] - own_a + 1, own_second = s_second[0];
  for (int e = threadIdx.x; e < G * (HD / 4); e += blockDim.x) {
    const int h = e % G, c4 = e / G;
    const size_t row = (size_t)m * a.n_q + (size_t)gg * G + h;
    const int R = R0 + h, r = R % C::ROWS, t = 1 + R / C::ROWS - tile0;
    const int shared_a = g >= 0 ? s_cta[t][0] : 0, n_shared = g >= 0 ? s_cta[t][1] - shared_a + 1 : 0, n = n_shared + n_own;
    const int shared_second = s_second[t];
    float ref = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = 0; b < n; b += kBatch) {
      float pr[kBatch], pl[kBatch];
      float4 pv[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int i = min(b + q, n - 1);
        const float *refs, *sums;
        const float4* at;
        if (i < n_shared) {
          const float* p = pa.pieces + (size_t)(2 * (shared_a + i) + (i == 0 ? shared_second : 0)) * pa.piece;
          refs = p + (size_t)pa.rows * HD + r;
          sums = refs + pa.rows;
          at = reinterpret_cast<const float4*>(p) + (size_t)c4 * pa.rows + r;
          if (n_shared == 1) {
            const size_t w = (size_t)m * G + h;
            refs = pa.whole_ref + (size_t)gg * RT + w;
            sums = pa.whole_l + (size_t)gg * RT + w;
            at = pa.whole + ((size_t)gg * (HD / 4) + c4) * RT + w;
          }
        } else {
          const int k = i - n_shared;
          const float* p = a.own_pieces + (size_t)(2 * (own_a + k) + (k == 0 ? own_second : 0)) * a.own_piece;
          refs = p + G * HD + h;
          sums = refs + G;
          at = reinterpret_cast<const float4*>(p + h * HD) + c4;
          if (n_own == 1) {
            refs = a.part_ref + row;
            sums = a.part_l + row;
            at = reinterpret_cast<const float4*>(a.part_o + row * HD) + c4;
          }
        }
        pr[q] = __ldcg(refs);
        pl[q] = __ldcg(sums);
        pv[q] = __ldcg(at);
      }
      float mx = ref;
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (b + q >= n || pl[q] == 0.f) pr[q] = -INFINITY;  // nothing attended to: the rest may hold anything
        mx = fmaxf(mx, pr[q]);
      }
      const float f = weight(ref, mx);
      sum *= f;
      o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (pr[q] == -INFINITY) continue;
        const float w = ex2(pr[q] - mx);
        sum += pl[q] * w;
        o.x += pv[q].x * w;
        o.y += pv[q].y * w;
        o.z += pv[q].z * w;
        o.w += pv[q].w * w;
      }
      ref = mx;
    }
    const float f = sum == 0.f ? 0.f : 1.0f / sum;
    *reinterpret_cast<uint2*>(a.o + row * HD + 4 * c4) = make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
    if (a.lse && c4 == 0) a.lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
  }
}

// The workspace behind paged attention's: the plan, the requests' own parts, the tiles that are not split, the pieces.
struct Layout {
  size_t plan, own_plan, own_o, own_ref, own_l, own_pieces, whole, whole_ref, whole_l, pieces, total;
  int piece, rows, own_piece;
};
Layout layout_of(int n_q, int n_kv, int hd, int M) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const int G = n_q / n_kv;
  Layout w;
  size_t at = up(paged_attn_workspace_bytes(G, hd));
  auto take = [&](size_t n) {
    const size_t was = at;
    at += up(n);
    return was;
  };
  const size_t heads = (size_t)M * n_q;
  w.rows = (int)std::min<size_t>(hd == 256 ? 128 : 256, ((size_t)M * G + 31) / 32 * 32);
  w.piece = w.rows * (hd + 2);
  w.plan = take(8 * ((size_t)M + 2));
  w.own_piece = (G * (hd + 2) + 3) / 4 * 4;
  w.own_plan = take(8 * ((size_t)M + 2));
  w.own_pieces = take((size_t)2 * kTailMaxCtas * w.own_piece * 4);
  w.own_o = take(heads * hd * 4);
  w.own_ref = take(heads * 4);
  w.own_l = take(heads * 4);
  w.whole = take(heads * hd * 4);
  w.whole_ref = take(heads * 4);
  w.whole_l = take(heads * 4);
  w.pieces = take((size_t)2 * kPrefixMaxCtas * w.piece * 4);
  w.total = at;
  return w;
}

template <int HD, bool FP8>
cudaError_t launch(const GroupedAttnArgs& args, cudaStream_t st) {
  using C = XCfg<HD, FP8>;
  EncodeTiled enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const int page = 1 << args.page_shift;
  CUtensorMap tm[2];
  for (int i = 0; i < 2; ++i) {  // the pages as rows of positions
    const cuuint64_t dims[2] = {(cuuint64_t)HD, (cuuint64_t)args.t * args.n_pages * (args.n_kv / args.t) * page};
    const cuuint64_t strides[1] = {(cuuint64_t)C::ROWB};
    const cuuint32_t box[2] = {(cuuint32_t)(C::INB / (FP8 ? 1 : 2)), (cuuint32_t)std::min(page, C::KS)}, es[2] = {1, 1};
    if (enc(&tm[i], FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<uint8_t*>(i ? args.v_pages : args.k_pages), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            C::INB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  PrefixArgs p{};
  p.a = args;
  const Layout w = layout_of(args.n_q, args.n_kv, HD, args.M);
  uint8_t* ws = reinterpret_cast<uint8_t*>(args.ws);
  auto f = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
  p.plan = reinterpret_cast<long long*>(ws + w.plan);
  p.a.part_o = f(w.own_o);
  p.a.part_ref = f(w.own_ref);
  p.a.part_l = f(w.own_l);
  p.a.own_plan = reinterpret_cast<long long*>(ws + w.own_plan);
  p.a.own_pieces = f(w.own_pieces);
  p.a.own_piece = w.own_piece;
  p.whole = reinterpret_cast<float4*>(ws + w.whole);
  p.whole_ref = f(w.whole_ref);
  p.whole_l = f(w.whole_l);
  p.pieces = f(w.pieces);
  p.piece = w.piece;
  p.rows = w.rows;
  auto kernel = prefix_attn_kernel<HD, FP8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // An ordinary launch: this kernel begins when all work before it is complete and visible.  The two that follow may begin
  // beside it, and read what the call was given without a wait of their own: a wait of a kernel ahead would order that
  // kernel's reads only.  (Launched dependent 2 us less; with a wait at the beginning of the other two 3 to 16 us more.)
  kernel<<<dim3(std::min(sm_count(), kPrefixMaxCtas)), dim3(C::kThreads), C::SMEM, st>>>(tm[0], tm[1], p);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_tail_attn(p.a, FP8 ? TP_FP8_E4M3 : TP_BF16, HD, st);
  if (e != cudaSuccess) return e;
  const int threads = std::min(256, (args.n_q / args.n_kv * HD / 4 + 31) / 32 * 32);
  e = launch_dependent(prefix_join_kernel<HD, FP8>, dim3((unsigned)args.M * args.n_kv), dim3(threads), 0, st, p);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t prefix_attn_workspace_bytes(int n_q, int n_kv, int hd, int M) { return layout_of(n_q, n_kv, hd, M).total; }

cudaError_t launch_prefix_attn(const GroupedAttnArgs& a, int kv_dtype, int hd, cudaStream_t st) {
  auto go = [&](auto fp8) {
    constexpr bool F = decltype(fp8)::value;
    return hd == 64 ? launch<64, F>(a, st) : hd == 128 ? launch<128, F>(a, st) : launch<256, F>(a, st);
  };
  return kv_dtype == TP_BF16 ? go(std::false_type{}) : go(std::true_type{});
}

}  // namespace tpx
