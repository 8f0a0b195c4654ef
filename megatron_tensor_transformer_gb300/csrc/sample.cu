// The next token of each row of logits from a given random number: temperature, top-k, top-p, min-p.
//
// With w_i = exp((x_i - max x) / T), ranks by (logit, then the lower id), a token e is kept if
//   fewer than top_k tokens are ahead of it,
//   of those within top_k, what is ahead of it weighs less than top_p of them all,
//   and w_e >= min_p;
// and the lowest id up to which the kept weights exceed u times their sum is chosen.
//
// Which token that is may hang on the last bits of a sum over the vocabulary, so the sums must not depend on how
// they are split: a weight is a whole number of 2^-44 and sums are 64-bit integers, exact in any order.
// A weight is 2^-E, E = (max - x) log2(e) / T held with 32 bits behind the point: the difference to the maximum and
// its product with log2(e) / T are each two fp32 (the rounded value and the rounding's rest), 2^-F of the fraction F
// a table of 64 and a cubic in what is left (|r| <= 2^-7): good to 2^-29 of the weight, 2^-31 on average.
#include "common.cuh"
#include "paged.h"
#include "tc_ptx.cuh"

namespace tpx {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kNT = 1024, kNW = kNT / 32;

// Orders as the logit does, -0 as +0.
__device__ __forceinline__ uint32_t order_of(float x) {
  uint32_t b = __float_as_uint(x);
  if (b == 0x80000000u) b = 0;
  return b >> 31 ? ~b : b | 0x80000000u;
}
// (logit, then the lower id): the greater the further ahead
__device__ __forceinline__ uint64_t key_of(float x, int id) { return (uint64_t)order_of(x) << 32 | (uint32_t)~id; }

struct Scale {  // of a row's exponents
  float top, hi, lo;
};
__device__ __forceinline__ uint64_t weight_of(float x, const Scale& s, const uint32_t* table) {
  if (x == -INFINITY) return 0;
  const float d = s.top - x, t = d - s.top, rest = (s.top - (d - t)) + (-x - t);  // d + rest is exact
  const float p = __fmul_rn(d, s.hi);  // rounded here: its rest goes to lo
  if (!(p < 46.f)) return 0;
  const float lo = fmaf(d, s.lo, __fmul_rn(rest, s.hi)) + fmaf(d, s.hi, -p);
  const float whole = floorf(p);
  long long e = ((long long)(int)whole << 32) + __float2uint_rn((p - whole) * 4294967296.f) + __float2int_rn(lo * 4294967296.f);
  if (e <= 0) return 1ull << 44;
  const uint32_t f = (uint32_t)e;
  const uint32_t w = table[f >> 26];
  const float z = (float)((int)(f & 0x3ffffffu) - (1 << 25)) * -1.6138637e-10f;  // - ln 2 / 2^32
  const float q = fmaf(fmaf(z, 1.f / 6.f, 0.5f), z * z, z);
  const uint32_t v = min(w + __float2int_rn((float)w * q), 1u << 31);
  return ((uint64_t)v << 13) >> (int)(e >> 32);
}

// One CTA per row, the row read again for each step of the searches: exact and slow.
__global__ void __launch_bounds__(kNT) sample_kernel(const SampleArgs a) {
  __shared__ uint32_t table[64];
  __shared__ uint64_t s_sum[kNW];
  __shared__ float s_top[kNW];
  const int tid = threadIdx.x, m = blockIdx.x, V = a.vocab;
  const float* x = a.logits + (int64_t)m * a.ldl;
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  if (tid < 64) table[tid] = (uint32_t)__double2ll_rn(exp2(31.0 - (tid + 0.5) / 64));
  auto block_sum = [&](uint64_t v) {  // to all threads
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    __syncthreads();
    if ((tid & 31) == 0) s_sum[tid >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < kNW; ++w) v += s_sum[w];
    return v;
  };
  float top = -INFINITY;
  int bad = 0;
  for (int i = tid; i < V; i += kNT) {
    top = fmaxf(top, x[i]);
    bad |= !(x[i] < INFINITY);
  }
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  bad = __syncthreads_or(bad);
  for (int w = 0; w < kNW; ++w) top = fmaxf(top, s_top[w]);

  const float T = a.temperature ? a.temperature[m] : 1.f, tp = a.top_p ? a.top_p[m] : 1.f,
              mp = a.min_p ? a.min_p[m] : 0.f, u = a.u[m];
  const int tk = T <= 0.f ? 1 : a.top_k ? a.top_k[m] : 0;
  if (bad || top == -INFINITY || T != T || tp != tp || mp != mp || u != u) {
    if (tid == 0) {
      a.ids[m] = -1;
      if (a.logprob) a.logprob[m] = NAN;
    }
    return;
  }
  const double t64 = T <= 0.f ? 1.0 : fmax((double)T, 0x1p-100), c = 1.4426950408889634 / t64;
  Scale s{top, (float)c, 0.f};
  s.lo = (float)(c - (double)s.hi);

  // The lowest key that is kept: the least t for which what lies above it (all of `from` and over) is less than lim.
  auto lowest = [&](uint64_t from, uint64_t lim, bool weights) {
    uint64_t lo = 0, hi = key_of(top, 0);  // above hi there is nothing
    while (lo < hi) {
      const uint64_t t = lo + (hi - lo) / 2;
      uint64_t v = 0;
      for (int i = tid; i < V; i += kNT) {
        const uint64_t k = key_of(x[i], i);
        if (k > t && k >= from) v += weights ? weight_of(x[i], s, table) : 1;
      }
      if (block_sum(v) < lim) hi = t;
      else lo = t + 1;
    }
    return lo;
  };
  auto sum_from = [&](uint64_t from) {
    uint64_t v = 0;
    for (int i = tid; i < V; i += kNT)
      if (key_of(x[i], i) >= from) v += weight_of(x[i], s, table);
    return block_sum(v);
  };
  // the lowest key of the first rank
  uint64_t from = 0;
  if (tk > 0 && tk < V) from = lowest(0, tk, false);
  if (tp < 1.f) {
    const uint64_t all = sum_from(from);
    const uint64_t p = tp <= 0.f ? 0 : (uint64_t)((double)tp * 0x1p64);  // exact from 2^-40 on
    const uint64_t lim = __umul64hi(p, all) + (p * all != 0);
    from = lowest(from, lim == 0 ? 1 : lim, true);
  }
  if (mp > 0.f) {
    // w >= mp is x >= top + T ln mp: the lowest fp32 that is not less
    const double lowest_x = (double)top + t64 * log((double)fminf(mp, 1.f));
    float b = __double2float_ru(lowest_x);
    from = max(from, (uint64_t)order_of(b) << 32);
  }
  const uint64_t all = sum_from(from);
  const uint64_t target = u < 0.f ? 0 : u >= 1.f ? all - 1 : __umul64hi((uint64_t)((double)u * 0x1p64), all);
  // the lowest id up to which the weights pass the target
  int lo = 0, hi = V - 1;
  while (lo < hi) {
    const int id = (lo + hi) / 2;
    uint64_t v = 0;
    for (int i = tid; i <= id; i += kNT)
      if (key_of(x[i], i) >= from) v += weight_of(x[i], s, table);
    if (block_sum(v) > target) hi = id;
    else lo = id + 1;
  }
  if (tid == 0) {
    a.ids[m] = lo;
    if (a.logprob) a.logprob[m] = (float)(((double)x[lo] - (double)top) / t64 - log((double)all * 0x1p-44));
  }
}

}  // namespace

cudaError_t launch_sample_tokens(const SampleArgs& a, cudaStream_t st) {
  const cudaError_t e = launch_dependent(sample_kernel, dim3((unsigned)a.M), dim3(kNT), 0, st, a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tpx
