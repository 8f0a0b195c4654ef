// The next token of each row of logits from a given random number: temperature, top-k, top-p, min-p.
//
// With w_i = exp((x_i - max x) / T), ranks by (logit, then the lower id), a token e is kept if
//   fewer than top_k tokens are ahead of it,
//   of those within top_k, what is ahead of it weighs less than top_p of them all,
//   and w_e >= min_p;
// and the lowest id up to which the kept weights exceed u times their sum is chosen.
//
// Which token that is may hang on the last bits of a sum over the vocabulary, so the sums must not depend on how
// they are split: a weight is a whole number of 2^-44 (of a power of two at or
// just above the largest) and sums are 64-bit integers, exact in any order.
// A weight is 2^-E, E good to 32 bits behind the point: the product of x with log2(e) / T is two fp32 (the rounded value
// and the rounding's rest), taken from a whole number so that nothing is lost; 2^-E is a table of 256 for the nearest
// 256th and a parabola in what is left: good to 2^-29 of the weight, 2^-31 on average.
//
// A row is shared by the CTAs of a cluster, which keep it in shared memory (from global again where it is too long) and join
// through distributed shared memory.  With a temperature or min-p alone one pass sums the weights.  Top-k and top-p look
// for the key (logit, then the lower id) of the last kept token by bins: a histogram of approximate weights (or of
// counts) says in which bin the border lies, a second pass sums the exact weights above it, checks that it does, and lists
// that bin's tokens, among which the first CTA finds the border.  Where they are too many to list (flat rows, ties) the
// bin is divided again by key.
//
// Measured (128256 tokens): one row with top-p 23 us (256 threads a CTA 30, 1024 29: seven barriers of the cluster, and code that
// is run once); 256 rows with a temperature and min-p 105 us, 1.3 TB/s, half of the issue slots; 1000 rows with top-p 886 us, 0.6 TB/s,
// 51% of the issue slots.  Bound by issue and by the barriers between the passes, of which the exact sums are the
// longest; two CTAs per SM overlap.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "paged.h"
#include "tc_ptx.cuh"

namespace tpx {

namespace {

namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kNT = 512, kPerSm = 2;                     // threads of a CTA, CTAs that an SM holds
constexpr int kMaxC = 8;                                 // CTAs of a row
constexpr int kBins = 1024;                              // of a division by key
constexpr float kUnit = 4096.f;                          // of the approximate weights
constexpr int kList = 256;                               // tokens that are listed
constexpr int kFew = kList;                              // top-k's tokens, up to which they are taken from a list
constexpr int kMostShared = 32 * 1024;                   // logits of a CTA that are kept in shared memory
constexpr float kLightest = 46.f;                        // exponent from which a weight is 0

// Orders as the logit does, -0 as +0.
__device__ __forceinline__ uint32_t order_of(float x) {
  uint32_t b = __float_as_uint(x);
  if (b == 0x80000000u) b = 0;
  return b >> 31 ? ~b : b | 0x80000000u;
}
// (logit, then the lower id): the greater the further ahead
__device__ __forceinline__ uint64_t key_of(float x, int id) { return (uint64_t)order_of(x) << 32 | (uint32_t)~id; }

// 2^(31 - j / 256)
__device__ const uint32_t kPowers[256] = {
    2147483648u, 2141676973u, 2135885998u, 2130110682u, 2124350982u, 2118606857u, 2112878262u, 2107165158u,
    2101467502u, 2095785251u, 2090118366u, 2084466803u, 2078830522u, 2073209480u, 2067603638u, 2062012954u,
    2056437387u, 2050876895u, 2045331439u, 2039800978u, 2034285470u, 2028784876u, 2023299156u, 2017828268u,
    2012372174u, 2006930832u, 2001504204u, 1996092249u, 1990694927u, 1985312200u, 1979944027u, 1974590370u,
    1969251188u, 1963926443u, 1958616096u, 1953320108u, 1948038440u, 1942771053u, 1937517909u, 1932278970u,
    1927054196u, 1921843549u, 1916646992u, 1911464486u, 1906295993u, 1901141476u, 1896000896u, 1890874216u,
    1885761398u, 1880662405u, 1875577199u, 1870505744u, 1865448001u, 1860403934u, 1855373507u, 1850356681u,
    1845353420u, 1840363688u, 1835387448u, 1830424663u, 1825475297u, 1820539314u, 1815616678u, 1810707353u,
    1805811301u, 1800928489u, 1796058879u, 1791202437u, 1786359126u, 1781528911u, 1776711757u, 1771907628u,
    1767116489u, 1762338305u, 1757573041u, 1752820662u, 1748081133u, 1743354420u, 1738640488u, 1733939301u,
    1729250827u, 1724575029u, 1719911875u, 1715261330u, 1710623359u, 1705997930u, 1701385007u, 1696784557u,
    1692196547u, 1687620943u, 1683057710u, 1678506817u, 1673968228u, 1669441912u, 1664927835u, 1660425963u,
    1655936265u, 1651458706u, 1646993254u, 1642539877u, 1638098541u, 1633669214u, 1629251865u, 1624846459u,
    1620452965u, 1616071351u, 1611701585u, 1607343634u, 1602997467u, 1598663052u, 1594340357u, 1590029350u,
    1585730000u, 1581442275u, 1577166143u, 1572901575u, 1568648537u, 1564406999u, 1560176931u, 1555958300u,
    1551751076u, 1547555228u, 1543370725u, 1539197537u, 1535035634u, 1530884983u, 1526745556u, 1522617322u,
    1518500250u, 1514394310u, 1510299473u, 1506215708u, 1502142985u, 1498081275u, 1494030547u, 1489990772u,
    1485961921u, 1481943963u, 1477936870u, 1473940611u, 1469955159u, 1465980482u, 1462016553u, 1458063343u,
    1454120821u, 1450188960u, 1446267730u, 1442357104u, 1438457051u, 1434567544u, 1430688553u, 1426820052u,
    1422962010u, 1419114401u, 1415277195u, 1411450365u, 1407633882u, 1403827719u, 1400031848u, 1396246240u,
    1392470869u, 1388705706u, 1384950723u, 1381205894u, 1377471191u, 1373746586u, 1370032052u, 1366327563u,
    1362633090u, 1358948606u, 1355274085u, 1351609500u, 1347954824u, 1344310030u, 1340675091u, 1337049980u,
    1333434672u, 1329829140u, 1326233356u, 1322647296u, 1319070932u, 1315504238u, 1311947188u, 1308399756u,
    1304861917u, 1301333643u, 1297814910u, 1294305692u, 1290805962u, 1287315695u, 1283834865u, 1280363448u,
    1276901417u, 1273448747u, 1270005413u, 1266571390u, 1263146652u, 1259731174u, 1256324931u, 1252927899u,
    1249540052u, 1246161366u, 1242791816u, 1239431376u, 1236080024u, 1232737732u, 1229404479u, 1226080238u,
    1222764986u, 1219458698u, 1216161350u, 1212872918u, 1209593378u, 1206322705u, 1203060876u, 1199807867u,
    1196563654u, 1193328213u, 1190101520u, 1186883552u, 1183674286u, 1180473697u, 1177281762u, 1174098458u,
    1170923762u, 1167757650u, 1164600099u, 1161451085u, 1158310587u, 1155178580u, 1152055042u, 1148939949u,
    1145833280u, 1142735011u, 1139645120u, 1136563583u, 1133490379u, 1130425485u, 1127368878u, 1124320536u,
    1121280436u, 1118248556u, 1115224875u, 1112209370u, 1109202018u, 1106202798u, 1103211687u, 1100228665u,
    1097253708u, 1094286796u, 1091327906u, 1088377016u, 1085434106u, 1082499153u, 1079572136u, 1076653033u,
};
struct Power {
  uint32_t value;
  float rounded;
};

// Of a row: its largest logit, log2(e) / T in two parts, and the whole number R that weights are held against: 2^(y - R),
// y = x log2(e) / T, so that R is at or just above the largest y.  R of kFar: y is too large for it, and weights are held
// against the largest itself.
struct Scale {
  float top, hi, lo;
  int whole;
  float above_top;  // 2^R over the largest weight: in [1, 2), about
};
constexpr int kFar = 1 << 30;
// (max - x) log2(e) / T rounded to fp32: monotone in x, as the keys are
__device__ __forceinline__ float exponent_of(float x, const Scale& s) { return __fmul_rn(s.top - x, s.hi); }
// Whole numbers come out of the mantissa of a sum with 1.5 2^23 units, and no conversion is needed (they share the
// exponentials' unit).
constexpr float kWhole = 12582912.f;
constexpr int kWholeBits = 0x4b400000;
// y of kFar aside, for an exponent below kLightest.
__device__ __forceinline__ uint64_t near_weight(float x, const Scale& s, const Power* table) {
  const float y = __fmul_rn(x, s.hi), k = y + kWhole / 256.f, near = k - kWhole / 256.f;
  const float rest = (y - near) + fmaf(x, s.lo, fmaf(x, s.hi, -y));
  const int d = s.whole * 256 + (kWholeBits - (8 << 23)) - __float_as_int(k);  // 256 (R - near)
  const float z = rest * 0.69314718f, q = fmaf(z * 0.5f, z, z);  // 2^rest = 1 + z + z^2 / 2, |z| below 2^-9.5
  const Power w = table[d & 255];
  const uint32_t v = w.value + (uint32_t)(__float_as_int(fmaf(w.rounded, q, kWhole)) - kWholeBits);
  return ((uint64_t)v << 13) >> (d >> 8 & 63);
}
__device__ __noinline__ uint64_t far_weight(float x, const Scale& s, const Power* table) {
  const float df = s.top - x, t = df - s.top, left = (s.top - (df - t)) + (-x - t);  // df + left is exact
  const float y = __fmul_rn(df, s.hi), k = y + kWhole / 256.f, near = k - kWhole / 256.f;
  const float rest = -((y - near) + (fmaf(df, s.lo, __fmul_rn(left, s.hi)) + fmaf(df, s.hi, -y)));
  const int d = __float_as_int(k) - (kWholeBits - (8 << 23));
  const float z = rest * 0.69314718f, q = fmaf(z * 0.5f, z, z);
  const Power w = table[d & 255];
  const uint32_t v = w.value + (uint32_t)(__float_as_int(fmaf(w.rounded, q, kWhole)) - kWholeBits);
  return ((uint64_t)v << 13) >> (d >> 8 & 63);
}
__device__ __forceinline__ uint64_t weight_of(float x, const Scale& s, const Power* table) {
  if (!(exponent_of(x, s) < kLightest)) return 0;  // (an infinite difference too)
  return s.whole != kFar ? near_weight(x, s, table) : far_weight(x, s, table);
}

// the larger of the two, NaN if x is one (fmaxf drops it)
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float logit_of(uint32_t order) {  // of order_of
  return __uint_as_float(order >> 31 ? order & 0x7fffffffu : ~order);
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
// 2^64 p for p in [0, 1), rounded down (exact from 2^-40 on)
__device__ __forceinline__ uint64_t frac64(float p) {
  const uint32_t b = __float_as_uint(p);
  const int e = (int)(b >> 23) - 86;  // p = mantissa 2^(e - 64)
  const uint64_t mant = (b & 0x7fffffu) | 0x800000u;
  return !(p > 0.f) || b < 0x800000u || e <= -24 ? 0 : e >= 0 ? mant << e : mant >> -e;
}
// p of all: rounded down and up
__device__ __forceinline__ uint64_t share_down(float p, uint64_t all) { return __umul64hi(frac64(p), all); }
__device__ __forceinline__ uint64_t share_up(float p, uint64_t all) {
  const uint64_t q = frac64(p);
  return __umul64hi(q, all) + (q * all != 0);
}

// A key as an edge: whether a token's reaches it.
struct Edge {
  float x;
  uint32_t id;
  __device__ __forceinline__ explicit Edge(uint64_t key)
      : x(key >> 32 ? logit_of((uint32_t)(key >> 32)) : -INFINITY), id((uint32_t)key) {}
  __device__ __forceinline__ bool reached(float y, int of) const { return y > x || (y == x && ~(uint32_t)of >= id); }
};

// A division of the keys into bins, the highest keys first: by the weight, or evenly by key from `high` down.
struct Bins {
  uint64_t low, high;  // keys [low, high] are divided, the others have no bin
  int shift;           // < 0: by the weight
};
// The bin, by the weight, of an exponent below kLightest: the nearest 64th.
constexpr int kPerOctave = 64, kOctaves = 16;            // octaves that are summed at a time, the last with all that follow
constexpr int kLast = (int)kLightest;                    // the last octave with a bin
__device__ __forceinline__ int nearest_64th(float p) {  // large for a large exponent and an infinite one
  return __float_as_int(fmaf(p, (float)kPerOctave, kWhole)) - kWholeBits;
}
// What the first CTA tells the others, and what it is told.
struct Shared {
  float top[kMaxC];
  uint32_t hist[kBins], fine[2][kMaxC][kPerOctave];  // of the search for top-k's border, and for top-p's: no CTA may still
  float octave[2][kMaxC][kOctaves];                  // be reading what another one writes; these, two sums in turn
  uint64_t key[kList], weight[kList];
  int listed;                    // tokens of the bin, of which the first kList are listed
  uint64_t above[kMaxC], in[kMaxC], all[kMaxC], least[kMaxC], most[kMaxC];  // of each CTA
  // (the answer to all is in above[0], what lies above the bin, and all[0], the limit: fields of their own took 1.5% longer)
  int bin, state;                // the border's bin; what to do next
  int ahead, behind, step;       // bins between which the border's is (the first CTA's, one thread's)
  uint64_t border;               // the lowest key that is kept
  Bins bins;
};
enum { kFound, kAgain, kDivide };  // the border is known; it lies in another bin; divide the bin

// Grid: M clusters of C CTAs.
__global__ void __launch_bounds__(kNT, kPerSm) sample_kernel(const SampleArgs a, int per_cta, int in_shared) {
  constexpr int kNW = kNT / 32;
  static_assert(kBins % kNT == 0, "bins per thread");
  extern __shared__ __align__(16) float s_row[];
  __shared__ Shared sh;
  __shared__ Power table[256];
  __shared__ uint32_t fine[kPerOctave];
  __shared__ uint64_t s_sum[kNW], s_above[kNW], s_sum2[kNW], s_sum3[kNW], s_least[kNW], s_most[kNW];
  __shared__ float s_top[kNW], s_scale[2], s_floor;
  __shared__ double s_inv, s_min;
  __shared__ int s_at;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), c = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, m = blockIdx.x / C, V = a.vocab;
  cl.barrier_arrive();  // all have begun where it is waited for: then their memory may be written
  tc::griddep_wait();
  tc::griddep_launch_dependents();  // after the wait: what follows may then rely on all work before this kernel
  if (tid < 256) table[tid] = Power{kPowers[tid], (float)kPowers[tid]};

  // The row from the 16-byte boundary at or before it on: place i holds id i - lead.  This CTA's places are
  // [i0, i1), in vectors of four; a place outside the row holds -inf.
  const float* row = a.logits + (int64_t)m * a.ldl;
  const int lead = (int)(reinterpret_cast<uintptr_t>(row) >> 2 & 3);
  row -= lead;
  const int own = in_shared ? per_cta : 0;  // behind the row: the threads' own sums
  const int places = (lead + V + 3) / 4 * 4, i0 = min(places, c * per_cta), i1 = min(places, i0 + per_cta);
  auto vector_at = [&](int i) {  // global memory
    if (i >= lead && i + 4 <= lead + V) return __ldcs(reinterpret_cast<const float4*>(row + i));
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i + k >= lead && i + k < lead + V ? row[i + k] : -INFINITY;
    return make_float4(v[0], v[1], v[2], v[3]);
  };
  const float T = a.temperature ? a.temperature[m] : 1.f, tp = a.top_p ? a.top_p[m] : 1.f,
              mp = a.min_p ? a.min_p[m] : 0.f, u = a.u[m];
  const int tk = T <= 0.f || mp > 1.f ? 1 : a.top_k ? a.top_k[m] : 0;  // no weight passes a min-p above 1: the first rank
  if (tid == kNT - 1) {  // 64-bit arithmetic is slow here: one thread's, beside the loads
    const double t64 = T <= 0.f ? 1.0 : fmax((double)T, 0x1p-100), scale = 1.4426950408889634 / t64;
    // An infinite temperature: the two parts add up to 0, but a difference times the first is small, not 0, so that one past
    // fp32's range (a masked logit) is infinite and weighs 0 here too.
    s_scale[0] = fmaxf((float)scale, 0x1p-149f);
    s_scale[1] = (float)(scale - (double)s_scale[0]);
    s_inv = 1.0 / t64;
    s_min = !(mp > 0.f) ? 0.0 : T < INFINITY ? t64 * log((double)fminf(mp, 1.f)) : -INFINITY;  // infinite: all weigh 1
  }
  float top = -INFINITY;
  {
    constexpr int kAhead = 4;
    for (int i = i0 + 4 * tid; i < i1; i += 4 * kNT * kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        v[k] = i + 4 * kNT * k < i1 ? vector_at(i + 4 * kNT * k) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        top = max_nan(max_nan(top, max_nan(v[k].x, v[k].y)), max_nan(v[k].z, v[k].w));
        if (in_shared && i + 4 * kNT * k < i1) *reinterpret_cast<float4*>(s_row + (i + 4 * kNT * k - i0)) = v[k];
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(kFull, top, o));
  if (lane == 0) s_top[warp] = top;
  if (tid == 0) sh.listed = 0;
  for (int b = tid; b < kBins; b += kNT) sh.hist[b] = 0;
  cl.barrier_wait();
  __syncthreads();
  if (warp == 0) {
    top = s_top[lane % kNW];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(kFull, top, o));
    if (lane < C) cl.map_shared_rank(&sh, lane)->top[c] = top;
  }
  cl.sync();
  top = sh.top[0];
  for (int r = 1; r < C; ++r) top = max_nan(top, sh.top[r]);

  if (!(top > -INFINITY && top < INFINITY) || T != T || tp != tp || mp != mp || u != u) {  // no distribution
    if (c == 0 && tid == 0) {
      a.ids[m] = -1;
      if (a.logprob) a.logprob[m] = NAN;
    }
    return;
  }
  const float y_top = __fmul_rn(top, s_scale[0]);
  const bool near = fabsf(y_top) < 8000.f;
  const Scale s{top, s_scale[0], s_scale[1], near ? (int)ceilf(y_top) : kFar, near ? ex2(ceilf(y_top) - y_top) : 1.f};

  // f(place, four logits) over the CTA's vectors
  auto each = [&](int from, int to, int step, auto f) {
    for (int i = from; i < to; i += step) f(i, in_shared ? *reinterpret_cast<const float4*>(s_row + (i - i0)) : vector_at(i));
  };
  auto key_at = [&](float x, int place) { return key_of(x, place - lead); };
  Shared* first = cl.map_shared_rank(&sh, 0);
  // Exact sums: each warp those of a run of vectors, so that they add up in the order of ids.
  const int vectors = (i1 - i0) / 4, per_warp = (vectors + kNW - 1) / kNW;
  const int v0 = min(vectors, warp * per_warp), v1 = min(vectors, v0 + per_warp);
  bool summed = false;  // s_above holds the warps' exact sums of all tokens kept so far above the border's bin, and
  int in_list = 0;      // sh.key and sh.weight (the first CTA's and this one's, at least) those in it

  int turn = 0;
  // Of the keys from `from` on: the lowest before which fewer than k of them lie (share < 0), or before which less than
  // `share` of their sum does.
  auto lowest = [&](uint64_t from, int k, float share) {
    const bool by_weight = share >= 0.f;
    Bins bins{from, ~0ull, -1};
    uint64_t base = 0, limit = k;  // what lies above the bins; by_weight: limit is known after the first sums
    const Edge low{from};
    auto bin_of = [&](float x, int place) {
      if (bins.shift >= 0) {
        const uint64_t key = key_at(x, place);
        return key >= bins.low && key <= bins.high ? (int)((bins.high - key) >> bins.shift) : -1;
      }
      const float p = exponent_of(x, s);
      return p < kLightest && low.reached(x, place - lead) ? nearest_64th(p) : -1;
    };
    auto bin_exponent = [&](int b) {  // by key: of a bin's highest key
      if (bins.shift < 0) return (float)b * (1.f / kPerOctave);
      return exponent_of(logit_of((uint32_t)((bins.high - ((uint64_t)b << bins.shift)) >> 32)), s);
    };
    const bool plain = from == 0;  // the usual case, in fewer steps
    // The first division, by the weight: the octave that holds the border from sums of a thread's own (one atomic a logit
    // took 26 cycles a warp), then its bins.  Every CTA comes to the same conclusion from the same numbers.
    {
      float* mine = s_row + own + tid;
      auto find = [&](float v, float goal, float& before) {  // the lane whose part of the sum holds goal, and what is before
        float upto = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float x = __shfl_up_sync(kFull, upto, o);
          if (lane >= o) upto += x;
        }
        const unsigned over = __ballot_sync(kFull, upto >= goal && v > 0.f), some = __ballot_sync(kFull, v > 0.f);
        const int l = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
        before = __shfl_sync(kFull, upto - v, l);
        return l;
      };
      float goal = 0.f, before;
      int octave;
#pragma unroll 1
      for (int begin = 0;; begin += kOctaves - 1) {  // nearly always one or two times
#pragma unroll
        for (int o = 0; o < kOctaves; ++o) mine[o * kNT] = 0.f;
        if (plain) {
          each(i0 + 4 * tid, i1, 4 * kNT, [&](int, float4 v4) {
            const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float p = exponent_of(v[q], s);
              const int o = min((nearest_64th(p) >> 6) - begin, kOctaves - 1);
              if (o >= 0) mine[o * kNT] += by_weight ? ex2(-p) : p < kLightest ? 1.f : 0.f;
            }
          });
        } else {
          each(i0 + 4 * tid, i1, 4 * kNT, [&](int i, float4 v4) {
            const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float p = exponent_of(v[q], s);
              if (!(p < kLightest) || !low.reached(v[q], i + q - lead)) continue;
              const int o = min((nearest_64th(p) >> 6) - begin, kOctaves - 1);
              if (o >= 0) mine[o * kNT] += by_weight ? ex2(-p) : 1.f;
            }
          });
        }
        __syncthreads();
        turn ^= 1;
        for (int o = warp; o < kOctaves; o += kNW) {
          float sum = 0.f;
          for (int t = lane; t < kNT; t += 32) sum += s_row[own + o * kNT + t];
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(kFull, sum, x);
          if (lane < C) cl.map_shared_rank(&sh, lane)->octave[turn][c][o] = sum;
        }
        if (tid < kPerOctave) fine[tid] = 0;
        cl.sync();
        float part = 0.f;
        if (lane < kOctaves)
          for (int r = 0; r < C; ++r) part += sh.octave[turn][r][lane];
        if (begin == 0) {
          float all = part;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) all += __shfl_xor_sync(kFull, all, x);
          if (!by_weight && all < (float)k) return from;  // fewer than k tokens have a weight: all are kept
          goal = by_weight ? all * share : (float)k;
        }
        octave = find(part, goal, before);
        goal -= before;
        if (octave < kOctaves - 1 || begin + kOctaves - 1 > kLast) {
          octave = min(begin + octave, kLast);
          break;
        }
      }
      if (plain) {
        each(i0 + 4 * tid, i1, 4 * kNT, [&](int, float4 v4) {
          const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float p = exponent_of(v[q], s), near = fmaf(p, (float)kPerOctave, kWhole);
            const unsigned b = (unsigned)(__float_as_int(near) - (kWholeBits + octave * kPerOctave));
            // 2^x = 1 + x ln 2 is near enough
            const float rest = fmaf(p, (float)kPerOctave, kWhole - near);
            const uint32_t n = (uint32_t)(__float_as_int(fmaf(rest, -0.69314718f / kPerOctave * kUnit, kWhole + kUnit)) - kWholeBits);
            if (b < kPerOctave) atomicAdd(&fine[b], by_weight ? n : 1u);
          }
        });
      } else {
        each(i0 + 4 * tid, i1, 4 * kNT, [&](int i, float4 v4) {
          const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float p = exponent_of(v[q], s);
            if (!(p < kLightest)) continue;
            const int b = nearest_64th(p);
            if (b / kPerOctave != octave || !low.reached(v[q], i + q - lead)) continue;
            const uint32_t n = by_weight ? __float2uint_rn(ex2(bin_exponent(b) - p) * kUnit) : 1u;
            if (n) atomicAdd(&fine[b % kPerOctave], n);
          }
        });
      }
      __syncthreads();
      for (int t = tid; t < C * kPerOctave; t += kNT)
        cl.map_shared_rank(&sh, t / kPerOctave)->fine[by_weight][c][t % kPerOctave] = fine[t % kPerOctave];
      cl.sync();
      // two bins per lane
      float two[2] = {0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int b = 2 * lane + q;
        uint32_t n = 0;
        for (int r = 0; r < C; ++r) n += sh.fine[by_weight][r][b];
        two[q] = !by_weight || n == 0 ? (float)n : (float)n * ex2(-bin_exponent(octave * kPerOctave + b)) * (1.f / kUnit);
      }
      const int l = find(two[0] + two[1], goal, before);
      const float first_of = __shfl_sync(kFull, two[0], l);
      const int b = octave * kPerOctave + 2 * l + (first_of > 0.f && before + first_of >= goal ? 0 : 1);
      __syncthreads();
      if (tid == 0) sh.bin = b;
      __syncthreads();
    }
    for (bool first_sums = true;;) {
      if (tid == 0) {
        sh.ahead = -1;
        sh.behind = bins.shift < 0 ? kLast * kPerOctave + 1 : kBins;
        sh.step = 1;
      }
      // Divided by key: what the bins hold, tokens, or roughly their weights in terms of the bin's heaviest (whole numbers, in
      // any order).
      if (bins.shift >= 0) {
        each(i0 + 4 * tid, i1, 4 * kNT, [&](int i, float4 v4) {
          const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int b = bin_of(v[q], i + q);
            if (b < 0) continue;
            uint32_t n = 1;
            if (by_weight) n = __float2uint_rn(ex2(bin_exponent(b) - exponent_of(v[q], s)) * kUnit);
            if (n) atomicAdd(&sh.hist[b], n);
          }
        });
        __syncthreads();
        if (c != 0) {
          for (int b = tid; b < kBins; b += kNT) {
            const uint32_t n = sh.hist[b];
            if (n) {
              atomicAdd(&first->hist[b], n);
              sh.hist[b] = 0;
            }
          }
        }
        cl.sync();
        if (c == 0) {  // the bin with the border, as far as these tell
          constexpr int kEach = kBins / kNT;
          uint64_t n[kEach], sum = 0;  // in units of 2^-24 of the bins' first weight
          const float p0 = bin_exponent(0);
#pragma unroll
          for (int q = 0; q < kEach; ++q) {
            const int b = tid * kEach + q;
            const uint32_t h = sh.hist[b];
            sh.hist[b] = 0;
            n[q] = !by_weight || h == 0 ? h : (uint64_t)((float)h * ex2(p0 - bin_exponent(b)) * (0x1p24f / kUnit));
            sum += n[q];
          }
          uint64_t before = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(kFull, before, o);
            if (lane >= o) before += x;
          }
          if (lane == 31) s_sum[warp] = before;
          before -= sum;
          if (tid == 0) sh.bin = kBins - 1;  // where none is found below: too few tokens, or rounding
          __syncthreads();
          for (int w = 0; w < warp; ++w) before += s_sum[w];
          uint64_t goal = limit - base;
          if (by_weight) goal = (uint64_t)((float)goal * (0x1p-20f * s.above_top * ex2(p0)));
          if (goal == 0) goal = 1;
#pragma unroll
          for (int q = 0; q < kEach; ++q) {
            if (before < goal && before + n[q] >= goal) atomicMin(&sh.bin, tid * kEach + q);
            before += n[q];
          }
          __syncthreads();
          if (tid < C) {
            const int bin = sh.bin;
            cl.map_shared_rank(&sh, tid)->bin = bin;
          }
        }
        cl.sync();
      }
      for (;;) {
        // The exact sums above the bin and in it, its keys' ends, and its tokens, listed as far as they fit.
        const int bin = sh.bin;
        uint64_t above = 0, in = 0, all = 0, least = ~0ull, most = 0;
        auto list = [&](float x, int place, uint64_t w) {
          const uint64_t key = key_at(x, place);
          in += w;
          least = min(least, key);
          most = max(most, key);
          const int at = atomicAdd(&sh.listed, 1);
          if (at < kList) {
            sh.key[at] = key;
            sh.weight[at] = w;
          }
        };
        if (plain && by_weight && bins.shift < 0 && bin < kLast * kPerOctave && s.whole != kFar) {
          each(i0 + 4 * (v0 + lane), i0 + 4 * v1, 128, [&](int i, float4 v4) {
            const float v[4] = {v4.x, v4.y, v4.z, v4.w};
            uint64_t w[4];
            int b[4];
            bool any = false;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float p = exponent_of(v[q], s);
              b[q] = nearest_64th(p);
              w[q] = near_weight(v[q], s, table);
              if (b[q] < bin) above += w[q];
              if (b[q] > bin && p < kLightest) all += w[q];
              any |= b[q] == bin;
            }
            if (!any) return;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (b[q] == bin) list(v[q], i + q, w[q]);
          });
        } else each(i0 + 4 * (v0 + lane), i0 + 4 * v1, 128, [&](int i, float4 v4) {
          const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int b = bin_of(v[q], i + q);
            const uint64_t w = by_weight ? weight_of(v[q], s, table) : 1;
            above += b >= 0 && b < bin ? w : 0;
            all += b > bin ? w : 0;
            if (b == bin) list(v[q], i + q, w);
          }
        });
        all += above + in;
        above = warp_sum(above);
        in = warp_sum(in);
        all = warp_sum(all);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          least = min(least, __shfl_xor_sync(kFull, least, o));
          most = max(most, __shfl_xor_sync(kFull, most, o));
        }
        if (lane == 0) {
          s_above[warp] = above;
          s_sum2[warp] = in;
          s_sum3[warp] = all;
          s_least[warp] = least;
          s_most[warp] = most;
        }
        __syncthreads();
        if (warp < 5) {  // one of the five per warp
          const uint64_t* part = warp == 0 ? s_above : warp == 1 ? s_sum2 : warp == 2 ? s_sum3 : warp == 3 ? s_least : s_most;
          uint64_t v = lane < kNW ? part[lane] : warp == 3 ? ~0ull : 0;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const uint64_t x = __shfl_xor_sync(kFull, v, o);
            v = warp < 3 ? v + x : warp == 3 ? min(v, x) : max(v, x);
          }
          uint64_t* to = warp == 0 ? first->above : warp == 1 ? first->in : warp == 2 ? first->all : warp == 3 ? first->least
                                                                                                             : first->most;
          if (lane == 0) to[c] = v;
        }
        if (c != 0) {  // what is listed goes behind what the first CTA has
          const int n = sh.listed;
          if (tid == 0) s_at = n ? atomicAdd(&first->listed, n) : 0;
          in_list = n;
          __syncthreads();
          for (int i = tid; i < min(n, kList - s_at); i += kNT) {
            first->key[s_at + i] = sh.key[i];
            first->weight[s_at + i] = sh.weight[i];
          }
          if (tid == 0) sh.listed = 0;
        }
        cl.sync();
        if (c == 0) {
          above = base;
          in = all = most = 0;
          least = ~0ull;
          for (int r = 0; r < C; ++r) {
            above += sh.above[r];
            in += sh.in[r];
            all += sh.all[r];
            least = min(least, sh.least[r]);
            most = max(most, sh.most[r]);
          }
          if (by_weight && first_sums) limit = max(uint64_t(1), share_up(share, all));
          const int listed = sh.listed;
          in_list = listed;
          // (where kList are listed, some may not be there)
          const int state = above >= limit || above + in < limit ? kAgain : listed >= kList ? kDivide : kFound;
          if (state == kAgain && tid == 0) {
            // The first sums are fp32 and good to some 2^-20 of all, less than many bins hold.  Where they miss the border's bin:
            // 1, 2, 4, .. bins on until it is passed, then halves of what is left.  (One after another took a thousand passes,
            // 7 to 14 ms for 64 rows, where one token weighs nearly top-p of all; now 0.2.)
            const int step = sh.step;
            (above >= limit ? sh.behind : sh.ahead) = bin;
            const int half = (sh.ahead + sh.behind) >> 1;
            sh.step = 2 * step;
            for (int r = 0; r < C; ++r)
              cl.map_shared_rank(&sh, r)->bin = above >= limit ? max(bin - step, half) : min(bin + step, half);
          }
          uint64_t lowest_kept = ~0ull;
          if (state == kFound) {  // a token is kept if what is ahead of it is below the limit
            for (int i = warp; i < listed; i += kNW) {
              const uint64_t key = sh.key[i];
              uint64_t ahead = 0;
              for (int j = lane; j < listed; j += 32) ahead += sh.key[j] > key ? sh.weight[j] : 0;
              if (above + warp_sum(ahead) < limit) lowest_kept = min(lowest_kept, key);
            }
          }
          __syncthreads();
          if (lane == 0) s_least[warp] = lowest_kept;
          __syncthreads();
          if (tid < C) {
#pragma unroll
            for (int w = 0; w < kNW; ++w) lowest_kept = min(lowest_kept, s_least[w]);
            Shared* to_sh = cl.map_shared_rank(&sh, tid);
            to_sh->state = state;
            to_sh->border = lowest_kept;
            const int bits = 64 - __clzll((long long)(most - least));
            to_sh->bins = Bins{least, most, max(0, bits - 10)};
            to_sh->above[0] = above;
            to_sh->all[0] = limit;
          }
          if (tid == 0) sh.listed = 0;
        }
        cl.sync();
        limit = sh.all[0];
        first_sums = false;
        if (sh.state == kFound) {
          summed = by_weight && bins.shift < 0;
          return sh.border;
        }
        if (sh.state == kDivide) {
          bins = sh.bins;
          base = sh.above[0];
          break;
        }
      }
    }
  };

  auto choose = [&](int id, float x, uint64_t w, uint64_t all) {
    a.ids[m] = id;
    if (a.logprob) {
      const double lw = s.whole != kFar ? (double)x * s_inv - s.whole * 0.6931471805599453 : ((double)x - (double)top) * s_inv;
      a.logprob[m] = w == all ? 0.f : (float)(lw - log((double)all * 0x1p-44));
    }
  };
  uint64_t from = 0;
  if (tk > 0 && tk < V) from = lowest(from, tk, -1.f);
  if (from != 0 && tk <= kFew) {
    // Few tokens are left, tk of them: the first CTA takes them all from a list, one per thread.  32 rows of 128256 with
    // top-k of 20, 128 and 256: 23, 25 and 29 us, with top-p 24, 27 and 40; 27 and 50 by the passes below.
    const Edge edge{from};
    each(i0 + 4 * tid, i1, 4 * kNT, [&](int i, float4 v4) {
      const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (!edge.reached(v[q], i + q - lead)) continue;
        const int at = atomicAdd(&sh.listed, 1);
        sh.key[min(at, kList - 1)] = key_at(v[q], i + q);
      }
    });
    __syncthreads();
    if (c != 0) {
      const int n = min(sh.listed, kFew);
      if (tid == 0) s_at = n ? atomicAdd(&first->listed, n) : 0;
      __syncthreads();
      for (int i = tid; i < min(n, kList - s_at); i += kNT) first->key[s_at + i] = sh.key[i];
    }
    cl.sync();  // the last use of another CTA's memory
    if (c != 0) return;
    const int n = min(sh.listed, kFew);
    const uint64_t key = tid < n ? sh.key[tid] : 0;
    const float x = logit_of((uint32_t)(key >> 32));
    const uint64_t w = tid < n ? weight_of(x, s, table) : 0;
    if (tid < n) sh.weight[tid] = w;
    __syncthreads();
    bool kept = tid < n;
    if (tp < 1.f && tid < n) {
      uint64_t ahead = 0, all = 0;
      for (int j = 0; j < n; ++j) {
        ahead += sh.key[j] > key ? sh.weight[j] : 0;
        all += sh.weight[j];
      }
      kept = ahead < max(uint64_t(1), share_up(fmaxf(tp, 0.f), all));
    }
    if (mp > 0.f) kept = kept && key >= uint64_t(order_of(__double2float_ru((double)top + s_min))) << 32;
    __syncthreads();
    if (tid < n && !kept) sh.weight[tid] = 0;
    __syncthreads();
    if (!kept) return;
    uint64_t before = 0, all = 0;  // by id: the lower half of a key falls as it rises
    for (int j = 0; j < n; ++j) {
      before += (uint32_t)sh.key[j] > (uint32_t)key ? sh.weight[j] : 0;
      all += sh.weight[j];
    }
    const uint64_t target = u >= 1.f ? all - 1 : share_down(u, all);
    if (target >= before && target < before + w) choose((int)~(uint32_t)key, x, w, all);
    return;
  }
  if (tp < 1.f) from = lowest(from, 0, fmaxf(tp, 0.f));
  const uint64_t border = from;
  if (mp > 0.f) {
    // w >= mp is x >= top + T ln mp: from the lowest fp32 that is not less
    if (tid == 0) s_floor = __double2float_ru((double)top + s_min);
    __syncthreads();
    from = max(from, uint64_t(order_of(s_floor)) << 32);
  }

  // The sums of the kept weights.
  const Edge edge{from};
  auto kept_sum = [&](int i, float4 v4) {
    const float v[4] = {v4.x, v4.y, v4.z, v4.w};
    uint64_t w = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (edge.reached(v[q], i + q - lead)) w += weight_of(v[q], s, table);
    return w;
  };
  __syncthreads();  // (s_sum may still be read)
  if (summed && from == border) {  // known but for the border's bin, which is listed
    if (tid < kNW) s_sum[tid] = s_above[tid];
    __syncthreads();
    if (tid < in_list && sh.key[tid] >= border) {
      const int place = (int)~(uint32_t)sh.key[tid] + lead;
      if (place >= i0 && place < i1)
        atomicAdd(reinterpret_cast<unsigned long long*>(&s_sum[(place - i0) / 4 / per_warp]), sh.weight[tid]);
    }
  } else {
    uint64_t mine = 0;
    if (from == 0 && s.whole != kFar) {
      each(i0 + 4 * (v0 + lane), i0 + 4 * v1, 128, [&](int, float4 v4) {
        const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint64_t w = near_weight(v[q], s, table);
          if (exponent_of(v[q], s) < kLightest) mine += w;
        }
      });
    } else {
      each(i0 + 4 * (v0 + lane), i0 + 4 * v1, 128, [&](int i, float4 v) { mine += kept_sum(i, v); });
    }
    mine = warp_sum(mine);
    if (lane == 0) s_sum[warp] = mine;
  }
  __syncthreads();
  if (warp == 0) {
    const uint64_t sum = warp_sum(lane < kNW ? s_sum[lane] : 0);
    if (lane < C) cl.map_shared_rank(&sh, lane)->in[c] = sum;
  }
  cl.sync();  // the last use of another CTA's memory
  uint64_t all = 0, before = 0;
  for (int r = 0; r < C; ++r) {
    if (r < c) before += sh.in[r];
    all += sh.in[r];
  }
  // the lowest id up to which the sum passes this
  const uint64_t target = u >= 1.f ? all - 1 : share_down(u, all);
  if (target < before || target >= before + sh.in[c]) return;
  // The run of the warp that holds it, a vector per thread.
  int holder = 0;
  for (; holder < kNW - 1 && target >= before + s_sum[holder]; ++holder) before += s_sum[holder];
  const int h0 = min(vectors, holder * per_warp), h1 = min(vectors, h0 + per_warp);
  __syncthreads();  // s_sum is written anew
  for (int base = h0; base < h1; base += kNT) {  // (once: a run is shorter than the CTA has threads, but for long rows)
    const int at = i0 + 4 * (base + tid);
    float4 v4 = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (base + tid < h1) v4 = in_shared ? *reinterpret_cast<const float4*>(s_row + (at - i0)) : vector_at(at);
    const uint64_t here = kept_sum(at, v4);
    uint64_t upto = here;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    uint64_t start = before + upto - here;
    for (int w = 0; w < kNW; ++w) {
      if (w < warp) start += s_sum[w];
      before += s_sum[w];
    }
    __syncthreads();
    if (target < start || target >= start + here) continue;
    const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (!edge.reached(v[q], at + q - lead)) continue;
      const uint64_t w = weight_of(v[q], s, table);
      if (target < start + w) {
        choose(at + q - lead, v[q], w, all);
        break;
      }
      start += w;
    }
  }
}

}  // namespace

cudaError_t launch_sample_tokens(const SampleArgs& a, cudaStream_t st) {
  // CTAs per row: as few as keep it in shared memory, and twice as many while each has an SM to itself (clusters do not
  // fill every SM, so up to 128 in all).  32000 tokens: 1 row 22 us with 2 CTAs and 17 with 8; 76 rows 24 with 2 and 36 with 4.
  int c = 1;
  auto per_cta = [&](int n) { return ((a.vocab + 3 + 3) / 4 + n - 1) / n * 4; };  // places, the row's lead among them
  while (c < kMaxC && (per_cta(c) > 16 * 1024 || ((int64_t)a.M * 2 * c <= 128 && per_cta(2 * c) >= 2048))) c *= 2;
  const int per = per_cta(c), in_shared = per <= kMostShared;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (kMostShared + kOctaves * kNT) * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.M * c);
  cfg.blockDim = dim3(kNT);
  cfg.dynamicSmemBytes = ((in_shared ? (size_t)per : 0) + kOctaves * kNT) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, sample_kernel, a, per, in_shared);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tpx
