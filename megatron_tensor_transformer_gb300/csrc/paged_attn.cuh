// What the attention kernels over a paged cache share: exponentials, operand descriptors, bounded waits, the split of
// a list of work over CTAs, and the positions that a request attends to by itself.
#pragma once
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "paged.h"
#include "tc_ptx.cuh"

namespace tpx {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoRef = -3.402823466e38f;  // no reference yet: fp32's lowest, which every finite score reaches (one
                                            // that only reaches it is rightly a weight of 1 under it)
constexpr int kP = 128;                    // positions per chunk: the rows of an MMA

// what a sum taken under reference m counts under the reference mx (0 where nothing was summed)
__device__ __forceinline__ float weight(float m, float mx) { return m == -INFINITY ? 0.f : ex2(m - mx); }

// Shared-memory operand descriptor: strides in bytes, layout 2 / 4 / 6 / 0 = 128 / 64 / 32-byte swizzle / none.
// K-major: `stride` between 8-row groups.  Transposed (rows of k): `stride` between groups of 8 k,
// `lead` between the blocks of a swizzle row's length along the other side.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride, uint32_t layout) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((lead >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((stride >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)layout << 61;
}
// two floats as e4m3 codes (x in the low byte), and back
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t v) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3));
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t v) { return __half22float2(e4m3x2_half2(v)); }

// 16 bytes of a row of q, which RP neighbouring lanes hold, as fp16: q / 2^(e - 127) below 2^15, e the exponent field of the
// row's largest value less 14 (both factors stay normal).  An infinity makes the row NaN, as its scores would.
template <int RP>
__device__ __forceinline__ uint4 q_as_fp16(const uint4& v, int& e) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0, h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) top = max(top, max((w[k] >> 7) & 0xffu, (w[k] >> 23) & 0xffu));
#pragma unroll
  for (int x = 1; x < RP; x <<= 1) top = max(top, __shfl_xor_sync(kFull, top, x));
  e = min(max((int)top, 15), 254) - 14;
  const float inv = top == 255u ? NAN : __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 x = __floats2half2_rn(bf16_lo(w[k]) * inv, bf16_hi(w[k]) * inv);
    h[k] = *reinterpret_cast<const uint32_t*>(&x);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// A role's bounded waits.  After one that runs out (it sets the error word) the producer issues no more copies and
// an issuing thread no more MMAs, and each waits, bounded again, for what it has in flight; the softmax warps
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

// Positions that a group of `size` rows reads once for all of them: the whole pages of its prefix.  0: none, or too few
// to matter to any row (a window ends before them all).
__device__ __forceinline__ int shared_len(const GroupedAttnArgs& a, int size, int prefix) {
  if (size < 2 || prefix < 0 || (long long)prefix > ((long long)a.max_pages << a.page_shift)) return 0;
  const int p = prefix >> a.page_shift << a.page_shift;
  return a.window > 0 && p > a.window ? 0 : p;
}
// The group of row m, -1: none (cu_groups in order).
__device__ __forceinline__ int group_of(const GroupedAttnArgs& a, int m) {
  int g = 0;
  for (int hi = a.n_groups; g < hi;) {  // the first whose end is behind m
    const int mid = (g + hi) >> 1;
    if (a.cu_groups[mid + 1] <= m) g = mid + 1;
    else hi = mid;
  }
  return g < a.n_groups && a.cu_groups[g] <= m ? g : -1;
}
// What request m of length n leaves to its group: all of the shared positions, or none.
__device__ __forceinline__ int left_to_group(const GroupedAttnArgs& a, int g, int n) {
  if (g < 0) return 0;
  const int p = shared_len(a, a.cu_groups[g + 1] - a.cu_groups[g], a.prefix_lens[g]);
  return n >= p && (a.window <= 0 || n <= a.window) ? p : 0;
}
// Whether groups i, i + step, .. lie in order within the batch (to be joined over the threads).
__device__ __forceinline__ bool groups_in_order(const GroupedAttnArgs& a, int i, int step) {
  bool ok = true;
  for (; i <= a.n_groups; i += step) {
    const int c = a.cu_groups[i];
    ok = ok && (i == 0 ? c >= 0 : c >= a.cu_groups[i - 1]) && c <= a.M;
  }
  return ok;
}

// The positions that a request attends to by itself, in chunks of SP.
template <int SP>
__device__ __forceinline__ Span own_span(const GroupedAttnArgs& a, int m, bool groups) {
  Span s = span_of(a, m);
  if (s.c0 == s.c1) return s;
  if (groups) s.lo = max(s.lo, left_to_group(a, group_of(a, m), s.n));
  s.c0 = s.lo / SP;
  s.c1 = s.lo == s.n ? s.c0 : (s.n - 1) / SP + 1;
  return s;
}

__device__ __forceinline__ long long quot(long long x, long long y) {  // x / y, both >= 0: a 64-bit division only if it must be
  return (x | y) >> 32 ? x / y : (long long)((uint32_t)x / (uint32_t)y);
}
// The same as a call, for code that a CTA runs once: there an instruction takes some 20 cycles until it is in the cache,
// and a division's are many.
__device__ __noinline__ long long quot_call(long long x, long long y) { return quot(x, y); }
__device__ __forceinline__ long long split_at(long long U, int nct, int i) { return quot(U * i, nct); }
__device__ __forceinline__ int owner(long long U, int nct, long long u) {
  return (int)quot((u + 1) * nct + U - 1, U) - 1;
}

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

}  // namespace

}  // namespace tpx
