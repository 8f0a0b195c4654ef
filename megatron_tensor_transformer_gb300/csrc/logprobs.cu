// Log probabilities of given tokens, the row's entropy, the token's rank and the top alternatives, in
// one pass over fp32 logits.
//
//   m = max x,  S = sum e^(x - m),  T = sum e^(x - m) (x - m):
//   ln P(v) = x_v - m - ln S,   entropy = ln S - T / S   (both terms >= 0: nothing cancels)
// with m, S, T running per thread in fp32 (when m grows by d, S shrinks by e^-d and T by the same after
// T += S (m_old - m_new)).  The rank counts the ids ahead of the given one, whose logit is read first.
//
// HBM-bound: 4 bytes a logit.  A row is shared by the 1, 2, 4 or 8 CTAs of a cluster, more the fewer
// rows there are; they join through distributed shared memory, so there is no workspace and one launch.
//
// Top alternatives: (logit, id) as one 64-bit key, the greater the further ahead, so ties go to the
// lower id.  A value is a candidate only if it reaches the bar, the k-th largest of the maxima that 32 or 64 groups
// of threads have seen so far: k values reach it, so no smaller one is among the k first.  The bar is
// taken anew after 1, 6 and 32 rounds, before the round's own values are looked at; of random values
// the 9 largest or so reach it for k = 8, the 31 largest for k = 20.  Each warp keeps its k best
// candidates, sorted across its lanes, inserting one at a time; at the end those that reach the last bar
// are ranked against each other, and the CTAs' k best in turn.  (Merging the warps' lists pairwise cost
// 32 rows 9 us, more than reading them.)
//
// Measured on one GB300, 128256 logits a row: 1900 rows 156 us without alternatives (92% of the measured
// copy's 6792 GB/s), 182 with one, 206 with 20 (70%: instructions issue in 75% of the cycles; 219 where the given tokens
// are random ids and not likely ones, so that more logits are compared with theirs one by one); 32 rows 7.2 us
// without, 10.8 with 8.  Short rows are a launch and the barriers: 2000 rows of 2000 logits 20 us, with 20
// alternatives 39.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "paged.h"
#include "tc_ptx.cuh"

namespace tpx {

namespace {

namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kNT = 512, kNW = kNT / 32, kMaxC = 8, kVec = 4;
static_assert(kNT == 64 * 8, "raise_bar takes 64 groups");


// the larger of the two, NaN if x is one (fmaxf drops it)
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

// Orders as (logit, then the lower id first); 0 is below every key of a number.
__device__ __forceinline__ uint64_t key_of(float x, int id) {
  uint32_t b = __float_as_uint(x);
  if (b == 0x80000000u) b = 0;  // -0 equals +0
  b = b >> 31 ? ~b : b | 0x80000000u;
  return (uint64_t)b << 32 | (uint32_t)(0x7fffffff - id);
}
__device__ __forceinline__ int key_id(uint64_t k) { return 0x7fffffff - (int)(uint32_t)k; }
__device__ __forceinline__ float key_logit(uint64_t k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float(b >> 31 ? b & 0x7fffffffu : ~b);
}

// Sums of a part of a row under its maximum (in units of the logits).  S is 0 where there is nothing but
// -inf, and NaN where there was a NaN or +inf (whose difference to the maximum is NaN), for good.
struct Part {
  float m, S, T;
};
__device__ __forceinline__ Part join(const Part& a, const Part& b) {
  if (a.S == 0.f) return b;
  if (b.S == 0.f) return a;
  const float m = fmaxf(a.m, b.m), da = a.m - m, db = b.m - m;
  const float fa = ex2(da * kLog2e), fb = ex2(db * kLog2e);
  // a part that weighs nothing adds nothing (its difference times its sum may be infinite)
  return {m, a.S * fa + b.S * fb, (fa > 0.f ? (a.T + a.S * da) * fa : 0.f) + (fb > 0.f ? (b.T + b.S * db) * fb : 0.f)};
}

struct Shared {
  Part part;
  int ahead;
  uint64_t top[32];
};

template <int C>
__global__ void __launch_bounds__(kNT, 2) logprobs_kernel(const LogprobsArgs a) {
  __shared__ Shared sh;
  __shared__ Part s_part[kNW];
  __shared__ int s_ahead[kNW];
  __shared__ uint64_t s_key[kNT];
  __shared__ __align__(16) float s_max[64];  // the groups' maxima
  __shared__ float s_bar;
  __shared__ int s_n;
  tc::griddep_wait();
  tc::griddep_launch_dependents();  // after the wait: what follows may then rely on all work before this kernel
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m = blockIdx.x / C, c = blockIdx.x % C, V = a.vocab, k = a.k;
  const float* x = a.logits + (int64_t)m * a.ldl;
  const int id = a.ids ? a.ids[m] : -1;
  const bool asked = id >= 0 && id < V;
  const float mine = asked ? x[id] : 0.f;

  // The row from its first 16-byte boundary on, in vectors of four; what is before and behind it goes one by one.
  const int lead = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / 4), nv = (V - lead) / 4;
  const int v0 = (int)((int64_t)nv * c / C), v1 = (int)((int64_t)nv * (c + 1) / C);
  const float4* xv = reinterpret_cast<const float4*>(x + lead);
  Part p{-INFINITY, 0.f, 0.f};
  int ahead = 0;
  uint64_t top = 0;
  float bar = -INFINITY;  // nothing below it is among the k first

  auto insert = [&](float val, int at, bool there) {  // whole warp: lane's value, if there
    const uint64_t key = there ? key_of(val, at) : 0;
    uint64_t kth = __shfl_sync(kFull, top, k - 1);
    unsigned cand = __ballot_sync(kFull, key > kth);
    while (cand) {
      const uint64_t nk = __shfl_sync(kFull, key, __ffs(cand) - 1);
      cand &= cand - 1;
      if (nk > kth) {
        const uint64_t up = __shfl_up_sync(kFull, top, 1);
        if (nk > top) top = lane == 0 || nk < up ? nk : up;
        kth = __shfl_sync(kFull, top, k - 1);
      }
    }
  };
  // 32 groups of 16 threads for k <= 24, else 64 of 8 (1900 rows, k = 20: 214.7 and 234.5 us; k = 32: 284.5 and 251.9)
  const bool small = k <= 24;
  auto ahead_of = [&](float v, int n) {  // how many of the first n maxima are ahead of this thread's, ties by place
    int r = 0;
#pragma unroll 8
    for (int i = 0; i < n; i += 4) {
      const float4 y4 = *reinterpret_cast<const float4*>(s_max + i);
      const float y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) r += y[j] > v || (y[j] == v && i + j < tid);
    }
    return r;
  };
  auto raise_bar = [&](float seen) {  // whole CTA; seen: the thread's maximum so far
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) seen = fmaxf(seen, __shfl_xor_sync(kFull, seen, o));
    if (small) {
      seen = fmaxf(seen, __shfl_xor_sync(kFull, seen, 8));
      if ((lane & 15) == 0) s_max[warp * 2 + (lane >> 4)] = seen;
    } else if ((lane & 7) == 0) {
      s_max[warp * 4 + (lane >> 3)] = seen;
    }
    __syncthreads();
    if (warp == 0 || (warp == 1 && !small)) {
      const float v = s_max[tid];
      if ((small ? ahead_of(v, 32) : ahead_of(v, 64)) == k - 1) s_bar = v;
    }
    __syncthreads();
    bar = s_bar;
  };
  // Ranks n keys of s_key, one per thread; the k first go to out, in order.
  auto rank = [&](int n, uint64_t* out) {
    if (tid < n) {
      const uint64_t key = s_key[tid];
      int r = 0;
      for (int i = 0; i < n; ++i) r += s_key[i] > key;
      if (r < k) out[r] = key;
    }
  };
  const int rounds = (v1 - v0 + kNT * kVec - 1) / (kNT * kVec);
  float4 q[kVec];
  auto load = [&](int r) {  // a vector that is not there holds -inf: no weight
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const int i = v0 + (r * kVec + u) * kNT + tid;
      q[u] = i < v1 ? __ldcs(xv + i) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
  };
  load(0);
  for (int r = 0; r < rounds; ++r) {
    const int i0 = v0 + r * kNT * kVec + tid;
    float v[kVec][4];
#pragma unroll
    for (int u = 0; u < kVec; ++u) v[u][0] = q[u].x, v[u][1] = q[u].y, v[u][2] = q[u].z, v[u][3] = q[u].w;
    if (r + 1 < rounds) load(r + 1);  // in flight while these are summed
    float mx[kVec], now = -INFINITY;
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      mx[u] = fmaxf(fmaxf(v[u][0], v[u][1]), fmaxf(v[u][2], v[u][3]));
      now = fmaxf(now, mx[u]);
    }
    if (now > p.m) {
      if (p.m != -INFINITY) {
        const float d = p.m - now, f = ex2(d * kLog2e);
        p.T = f > 0.f ? (p.T + p.S * d) * f : 0.f;  // as in join()
        p.S *= f;
      }
      p.m = now;
    }
    const float base = p.m == -INFINITY ? 0.f : p.m;  // only -inf so far: every weight is 0
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float d = max_nan(v[u][j] - base, -1e4f), e = ex2(d * kLog2e);
        p.S += e;
        p.T += e * d;
      }
      if (mx[u] >= mine && i0 + u * kNT < v1) {
        const int at = lead + 4 * (i0 + u * kNT);
#pragma unroll
        for (int j = 0; j < 4; ++j) ahead += v[u][j] > mine || (v[u][j] == mine && at + j < id);
      }
    }
    if (k > 0) {
      if (r == 0 || r == 5 || r == 31) raise_bar(p.m);
      if (__any_sync(kFull, now >= bar)) {
#pragma unroll
        for (int u = 0; u < kVec; ++u) {
          const bool there = i0 + u * kNT < v1;
          if (!__any_sync(kFull, there && mx[u] >= bar)) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool in = there && v[u][j] >= bar;
            if (__any_sync(kFull, in)) insert(v[u][j], lead + 4 * (i0 + u * kNT) + j, in);
          }
        }
      }
    }
  }
  if (c == 0 && warp == 0) {  // the ends, at most three values each
    const int at = lane < 4 ? lane : lead + 4 * nv + lane - 4;
    const bool there = lane < 4 ? lane < lead : lane < 8 && at < V;
    const float v = there ? x[at] : -INFINITY;
    if (there) {
      p = join(p, Part{v, v == -INFINITY ? 0.f : v < INFINITY ? 1.f : NAN, 0.f});
      ahead += v > mine || (v == mine && at < id);
    }
    if (k > 0) insert(v, at, there);
  }

  // the warp's, the CTA's, the cluster's
  auto join_lanes = [&](int n) {
    for (int o = n / 2; o > 0; o >>= 1) {
      const Part q{__shfl_xor_sync(kFull, p.m, o), __shfl_xor_sync(kFull, p.S, o), __shfl_xor_sync(kFull, p.T, o)};
      p = join(p, q);
      ahead += __shfl_xor_sync(kFull, ahead, o);
    }
  };
  join_lanes(32);
  if (lane == 0) {
    s_part[warp] = p;
    s_ahead[warp] = ahead;
  }
  if (tid == 0) s_n = 0;
  if (tid < 32) sh.top[tid] = 0;
  __syncthreads();
  if (k > 0) {
    const bool in = lane < k && top != 0 && key_logit(top) >= bar;
    const unsigned who = __ballot_sync(kFull, in);
    int at = lane == 0 && who ? atomicAdd(&s_n, __popc(who)) : 0;
    at = __shfl_sync(kFull, at, 0) + __popc(who & ((1u << lane) - 1));
    if (in) s_key[at] = top;
    __syncthreads();
    rank(s_n, sh.top);
    __syncthreads();
  }
  if (warp == 0) {
    p = s_part[lane % kNW];
    ahead = s_ahead[lane % kNW];
    join_lanes(kNW);
    if (lane == 0) {
      sh.part = p;
      sh.ahead = ahead;
    }
  }
  if (C > 1) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    if (c == 0 && warp < C) {  // warp r brings CTA r's
      const Shared* o = cl.map_shared_rank(&sh, warp);
      if (lane < k) s_key[warp * k + lane] = o->top[lane];
      if (lane == 0) {
        s_part[warp] = o->part;
        s_ahead[warp] = o->ahead;
      }
    }
    cl.sync();  // the others' shared memory is read until here
    if (c != 0) return;
    __syncthreads();
    if (k > 0) {
      rank(C * k, sh.top);
      __syncthreads();
    }
    if (warp == 0) {
      p = s_part[lane % C];
      ahead = s_ahead[lane % C];
      join_lanes(C);
    }
  }
  if (warp != 0) return;
  if (lane < k) top = sh.top[lane];
  const bool none = !(p.S > 0.f);
  const float lnS = logf(p.S);
  if (lane == 0) {
    if (a.logprob) a.logprob[m] = !asked ? 0.f : none ? NAN : mine - p.m - lnS;
    if (a.rank) a.rank[m] = !asked || none ? 0 : ahead + 1;
    if (a.entropy) a.entropy[m] = none ? NAN : lnS - p.T / p.S;
  }
  if (lane < k) {
    a.top_logprob[(size_t)m * k + lane] = none ? NAN : key_logit(top) - p.m - lnS;
    a.top_id[(size_t)m * k + lane] = none ? -1 : key_id(top);
  }
}

template <int C>
cudaError_t launch(const LogprobsArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.M * C);
  cfg.blockDim = dim3(kNT);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, logprobs_kernel<C>, a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobsArgs& a, cudaStream_t st) {
  // CTAs per row: two if that is at most one per SM over all rows, four and eight up to 256 in all, while each
  // still has 4 vectors per thread.  With 1, 2, 4, 8 CTAs and 8 alternatives of 128256 logits, 32 rows take 21.0,
  // 16.2, 11.5, 10.8 us, 64 rows 21.9, 16.9, 15.7, 20.8, 76 rows 22.2, 17.1, 22.5, 27.7, 128 rows 22.4, 23.9, 29.3,
  // 39.4: a second CTA on some SMs takes them nearly as long again.  With 8 alternatives the rule is within 12% of the
  // best of these at 2000, 8000, 16000 and 64000 logits for 1 to 200 rows, and at 32000 for 48 rows and more; one row
  // of 32000 takes 7.7 us where four CTAs take 6.5, 16 rows 8.2 and 7.0.
  int c = 1;
  while (c < kMaxC && (int64_t)a.M * 2 * c <= (c == 1 ? 152 : 256) && a.vocab / (2 * c) >= 4 * 4 * kNT) c *= 2;
  return c == 1 ? launch<1>(a, st) : c == 2 ? launch<2>(a, st) : c == 4 ? launch<4>(a, st) : launch<8>(a, st);
}

}  // namespace tpx
