// Rotary positions on the QKV output, in place or on the way into the paged cache.
//
// The angle of pair i at position p is p * f_i.  In fp32 that product alone is off by 2^-24 p f_i
// radians (0.06 at p = 10^6), so it is taken in turns as a 64-bit binary fraction: p * step_i modulo
// 2^64, whose wrap-around is the reduction modulo whole turns.  The nearest quarter turn is
// split off as an integer and the rest, at most 1/8 turn, goes to sincospi in fp32: cos and sin are
// good to about an fp32 ulp at every position, and no 64-bit floating point is used.
//
// HBM-bound: each element is read and written once.  A thread holds 16 elements of a head, eight
// whole pairs as two 16-byte vectors (dims 8i.. and rot/2 + 8i.. for the half layout, 16i.. and
// 16i + 8.. for the interleaved one); the block is (hd / 16) x heads.  The cos and sin of a token
// are computed once per CTA, into shared memory, and shared by its heads.
// The heads of both tokens of a CTA are dealt to its threads at once (token by token, 80 heads took
// three passes of 32, the last one half empty: 61.5 us).
// Measured on one GB300: 8192 rows of 64 q and 8 kv heads of 128 into bf16 pages 56.5 us, 5.94 TB/s (a plain
// copy of as many bytes 50.0 us, the append without turning 52.9), rotated in the QKV order 56.0, in place 54.9; 32
// rows 2.6 us.  Bound by HBM and, beside it, by the angles and the turning.  Into e4m3 pages, 32 and 8 heads, half of
// each turned: 1 row 3.1 us, 608 rows 4.6, 1003 6.3, 8192 44.6 (61% of the copy's rate).  Of the 44.6 the turning is
// 6.3, the divides 2.7 and the coding with them 3.6; at six CTAs per SM instead of four, with fewer registers, 8192
// rows take 38.7 and 1003 rows 8.7.
#include "common.cuh"
#include "paged.h"
#include "tc_ptx.cuh"

#include <algorithm>

namespace tpx {

namespace {

enum { SINK_QKV = 0, SINK_BF16 = 1, SINK_E4M3 = 2 };

constexpr int kTok = 2;  // tokens per CTA at most

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = bf16_lo(w[j]);
    x[2 * j + 1] = bf16_hi(w[j]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// e4m3 codes of x / s, RNE satfinite (a NaN stays one)
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * j], s), __fdiv_rn(x[2 * j + 1], s)),
                                                __NV_SATFINITE, __NV_E4M3);
    w[j >> 1] |= c << (16 * (j & 1));
  }
  return make_uint2(w[0], w[1]);
}

// grid (token groups, head groups), block (hd / 16, heads a pass)
template <int SINK>
__global__ void __launch_bounds__(256, SINK == SINK_E4M3 ? 4 : 6) rope_kernel(const __grid_constant__ RopeArgs a, int toks, int heads) {
  __shared__ __align__(16) float cs[kTok][2][128];
  tc::griddep_wait();
  tc::griddep_launch_dependents();  // after the wait: what follows may then rely on all work before this kernel
  const int m0 = blockIdx.x * toks, nt = min(toks, a.M - m0), half = a.rope.rot_dim / 2;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthr = blockDim.x * blockDim.y;
  if (SINK != SINK_QKV && a.counters && blockIdx.x == 0 && blockIdx.y == 0)
    for (int j = tid; j < kPagedCounters; j += nthr) a.counters[j] = 0u;
  for (int j = tid; j < nt * half; j += nthr) {
    const int k = j / half, i = j % half;
    const uint64_t turn = (uint64_t)(int64_t)a.positions[m0 + k] * a.rope.step[i];
    const uint64_t near = turn + (1ull << 61);  // + 1/8 turn: the quarter it lies nearest to is its top two bits
    const int quarter = (int)(near >> 62);
    const int64_t rest = (int64_t)((near & ((1ull << 62) - 1)) - (1ull << 61));  // [-1/8, 1/8) turn
    float sn, cn;
    sincospif((float)rest * 0x1p-63f, &sn, &cn);
    const float c = quarter & 1 ? (quarter & 2 ? sn : -sn) : (quarter & 2 ? -cn : cn);
    const float s = quarter & 1 ? (quarter & 2 ? -cn : cn) : (quarter & 2 ? -sn : sn);
    cs[k][0][i] = c * a.rope.mscale;
    cs[k][1][i] = s * a.rope.mscale;
  }
  __syncthreads();
  const int hd = a.hd, per = (a.n_q + 2 * a.n_kv) / a.t, nqs = a.n_q / a.t, nkvs = a.n_kv / a.t, all = per * a.t;
  const unsigned per_inv = 0xffffffffu / per + 1;  // h / per as a high product: exact while all * per < 2^32
  const int i = threadIdx.x;
  const bool turned = 8 * i < half;
  // the thread's two vectors within the head
  const bool split = turned && a.rope.layout == TP_ROPE_HALF;
  const int d0 = split ? 8 * i : 16 * i, d1 = split ? half + 8 * i : 16 * i + 8;
  const int h0 = blockIdx.y * heads, nh = min(all - h0, heads);
  int slots[kTok] = {};
  if (SINK != SINK_QKV)
    for (int k = 0; k < nt; ++k) slots[k] = a.slots[m0 + k];
  for (int e = threadIdx.y; e < nt * nh; e += blockDim.y) {
    static_assert(kTok == 2, "k is 0 or 1");
    const int k = e >= nh, h = h0 + e - (k ? nh : 0), m = m0 + k;
    const __nv_bfloat16* row = a.qkv + (size_t)m * all * hd;
    int slot = 0;
    bool kept = true;
    if (SINK != SINK_QKV) {
      slot = k ? slots[1] : slots[0];
      kept = slot >= 0 && (slot >> a.page_shift) < a.n_pages;
    }
    const int sh = (int)__umulhi((unsigned)h, per_inv), l = h - sh * per;
    const bool is_q = l < nqs, is_v = l >= nqs + nkvs;
    if (SINK == SINK_QKV && is_v && a.q_out == a.qkv) continue;  // in place
    if (SINK != SINK_QKV && !is_q && !kept) continue;
    const uint4 u0 = *reinterpret_cast<const uint4*>(row + (size_t)h * hd + d0);
    const uint4 u1 = *reinterpret_cast<const uint4*>(row + (size_t)h * hd + d1);
    float x[8], y[8];
    uint4 o0 = u0, o1 = u1;
    const bool turn_it = turned && !is_v;
    unpack8(u0, x);
    unpack8(u1, y);
    if (turn_it) {
      float c[8], s[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 cv = *reinterpret_cast<const float4*>(&cs[k][0][8 * i + 4 * j]);
        const float4 sv = *reinterpret_cast<const float4*>(&cs[k][1][8 * i + 4 * j]);
        c[4 * j] = cv.x, c[4 * j + 1] = cv.y, c[4 * j + 2] = cv.z, c[4 * j + 3] = cv.w;
        s[4 * j] = sv.x, s[4 * j + 1] = sv.y, s[4 * j + 2] = sv.z, s[4 * j + 3] = sv.w;
      }
      if (split) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = x[j], q = y[j];
          x[j] = p * c[j] - q * s[j];
          y[j] = q * c[j] + p * s[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = x[2 * j], q = x[2 * j + 1], u = y[2 * j], v = y[2 * j + 1];
          x[2 * j] = p * c[j] - q * s[j];
          x[2 * j + 1] = q * c[j] + p * s[j];
          y[2 * j] = u * c[4 + j] - v * s[4 + j];
          y[2 * j + 1] = v * c[4 + j] + u * s[4 + j];
        }
      }
      o0 = pack8(x);
      o1 = pack8(y);
    }
    if (SINK == SINK_QKV || is_q) {
      __nv_bfloat16* out = SINK == SINK_QKV ? a.q_out + ((size_t)m * all + h) * hd
                                            : a.q_out + ((size_t)m * a.n_q + sh * nqs + l) * hd;
      *reinterpret_cast<uint4*>(out + d0) = o0;
      *reinterpret_cast<uint4*>(out + d1) = o1;
    } else {
      const int g = is_v ? l - nqs - nkvs : l - nqs;  // kv head within the shard
      const size_t page = (size_t)sh * a.n_pages + (slot >> a.page_shift);
      const size_t at = (((page * nkvs + g) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) * hd;
      if (SINK == SINK_BF16) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_v ? a.v_pages : a.k_pages) + at;
        *reinterpret_cast<uint4*>(out + d0) = o0;
        *reinterpret_cast<uint4*>(out + d1) = o1;
      } else {
        const float* scale = is_v ? a.v_scale : a.k_scale;
        const float sc = scale ? scale[sh * nkvs + g] : 1.0f;
        uint8_t* out = static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages) + at;
        *reinterpret_cast<uint2*>(out + d0) = codes8(x, sc);
        *reinterpret_cast<uint2*>(out + d1) = codes8(y, sc);
      }
    }
  }
}

template <int SINK>
cudaError_t launch(const RopeArgs& a, cudaStream_t st) {
  const int tx = a.hd / 16, ty = 256 / tx, all = a.n_q + 2 * a.n_kv;
  // Few tokens: one token and one pass of heads per CTA, to fill the SMs; many: kTok tokens, all heads (with 1 and
  // 2 per CTA 8192 rows into bf16 pages took 59.5 and 56.5 us, 1003 rows into e4m3 pages 7.3 and 6.2; 3 and 4,
  // which take a division per head, 57.7 and 61.6, 8.1 and 6.8).
  const bool many = (int64_t)a.M * ((all + ty - 1) / ty) > 4 * 152;
  const int toks = many ? kTok : 1, heads = many ? all : ty;
  const cudaError_t e = launch_dependent(rope_kernel<SINK>, dim3(a.M / toks + (a.M % toks != 0), (all + heads - 1) / heads),
                                         dim3(tx, ty), 0, st, a, toks, heads);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) { return launch<SINK_QKV>(a, st); }
cudaError_t launch_rope_append(const RopeArgs& a, int kv_dtype, cudaStream_t st) {
  return kv_dtype == TP_BF16 ? launch<SINK_BF16>(a, st) : launch<SINK_E4M3>(a, st);
}

}  // namespace tpx
