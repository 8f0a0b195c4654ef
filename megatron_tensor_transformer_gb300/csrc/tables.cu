// Block tables and slots of a serving step from the requests' lengths, in one launch.
//
// Two exclusive sums over the requests give everything: of the new rows (where a request's tokens
// lie in the batch) and of the new pages (where its pages lie in the free list).  Every CTA takes
// both sums over all requests (a contiguous run of requests per thread, then a block scan: 8 bytes
// read per request, from L2 after the first CTA), so no CTA waits for another; then the CTAs share
// the rows.  A row finds its request by a running maximum over marks that the requests leave at
// their first row of a slice, so a prompt of many rows costs no more per row than many requests of
// one.  The sums are 64-bit: lengths are device data and may be anything.
// Latency-bound (a few KB to a MB): 256 requests of one token 4.3 us on one GB300, 37 prompts of 144 thousand
// rows in all 4.8 us.
#include "common.cuh"
#include "paged.h"
#include "tc_ptx.cuh"

#include <algorithm>

namespace tpx {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// Block-wide exclusive sum (total in *sum); part: one word per warp.  Ends with every thread past its reads.
template <int NT>
__device__ long long block_scan(long long v, long long* part, long long* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const long long p = part[w];
    if (w < warp) before += p;
    all += p;
  }
  __syncthreads();
  *sum = all;
  return before + incl - v;
}

struct Req {
  long long rows, need;  // its rows in the batch; the pages it needs if its rows are at `first`
  int len;
  bool ok;
};

// Request m with its first row at `first`.
__device__ __forceinline__ Req request(const TablesArgs& a, int m, long long first) {
  const int len = a.lens[m], add = a.add[m];
  const long long end = (long long)len + add, pm = (1 << a.page_shift) - 1;
  Req r{add > 0 ? add : 0, 0, len, false};
  r.ok = len >= 0 && add >= 0 && end <= min((long long)a.max_pages << a.page_shift, 0x7fffffffll) &&
         first + r.rows <= a.rows;
  if (r.ok) r.need = ((end + pm) >> a.page_shift) - ((len + pm) >> a.page_shift);
  return r;
}

// NT threads; each slice of NT rows has one thread per row.
template <int NT>
__global__ void __launch_bounds__(NT) tables_kernel(const TablesArgs a) {
  __shared__ long long part[NT / 32];
  __shared__ int mark[NT], wmax[NT / 32];
  __shared__ int s_m[NT], s_len[NT];
  __shared__ long long s_first[NT], s_base[NT];  // the request's first row; its first page in the free list
  __shared__ bool s_in[NT];                      // whether it is served (it may be without pages left: s_base is then unused)
  tc::griddep_wait();
  tc::griddep_launch_dependents();  // after the wait: what follows may then rely on all work before this kernel
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = a.M / NT + (a.M % NT != 0), m0 = min(a.M, tid * per), m1 = m0 + min(per, a.M - m0);
  const long long head = a.head ? *a.head : 0;
  const long long left = head >= 0 && head <= a.n_free ? a.n_free - head : 0;

  long long rows_here = 0, total_rows, total_need;
  for (int m = m0; m < m1; ++m) rows_here += max(a.add[m], 0);
  const long long first0 = block_scan<NT>(rows_here, part, &total_rows);
  long long need_here = 0, first = first0;
  for (int m = m0; m < m1; ++m) {
    const Req r = request(a, m, first);
    need_here += r.need;
    first += r.rows;
  }
  const long long need0 = block_scan<NT>(need_here, part, &total_need);

  if (blockIdx.x == 0) {
    long long taken = 0, refused = 0, need = need0;
    first = first0;
    for (int m = m0; m < m1; ++m) {
      const Req r = request(a, m, first);
      need += r.need;
      const bool in = r.ok && (r.need == 0 || need <= left);
      if (in) taken += r.need;
      else ++refused;
      a.lens_out[m] = in ? r.len + (int)r.rows : r.len;
      a.cu_rows[m] = (int)min(first, 0x7fffffffll);
      first += r.rows;
    }
    long long all_taken, all_refused;
    block_scan<NT>(taken, part, &all_taken);
    block_scan<NT>(refused, part, &all_refused);
    if (tid == 0) {
      a.cu_rows[a.M] = (int)min(total_rows, 0x7fffffffll);
      a.counts[0] = (int)(head + all_taken);
      a.counts[1] = (int)min(total_rows, 0x7fffffffll);
      a.counts[2] = (int)all_refused;
    }
  }

  const int pmask = (1 << a.page_shift) - 1;
  for (long long r0 = (long long)blockIdx.x * NT; r0 < a.rows; r0 += (long long)gridDim.x * NT) {
    mark[tid] = -1;
    __syncthreads();
    if (first0 < r0 + NT && first0 + rows_here > r0) {  // some of this thread's requests have rows here
      long long need = need0;
      first = first0;
      for (int m = m0; m < m1; ++m) {
        const Req r = request(a, m, first);
        if (r.rows > 0 && first < r0 + NT && first + r.rows > r0) {
          const int i = (int)(max(first, r0) - r0);
          mark[i] = i;
          s_m[i] = m;
          s_len[i] = r.len;
          s_first[i] = first;
          s_base[i] = head + need;
          s_in[i] = r.ok && (r.need == 0 || need + r.need <= left);
        }
        need += r.need;
        first += r.rows;
      }
    }
    __syncthreads();
    int i = mark[tid];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, i, o);
      if (lane >= o) i = max(i, u);
    }
    if (lane == 31) wmax[warp] = i;
    __syncthreads();
    for (int w = 0; w < warp; ++w) i = max(i, wmax[w]);
    const long long row = r0 + tid;
    if (row < a.rows) {
      int pos = 0, slot = -1;
      if (row < total_rows) {
        const int m = s_m[i], len = s_len[i];
        const long long base = s_base[i];
        pos = (int)((unsigned)len + (unsigned)(row - s_first[i]));
        if (s_in[i]) {
          const int pg = pos >> a.page_shift, fresh = pg - (int)(((long long)len + pmask) >> a.page_shift);
          int* entry = a.table + (size_t)m * a.table_stride + pg;
          const int id = fresh >= 0 ? a.free_pages[base + fresh] : *entry;
          if (fresh >= 0 && (pos & pmask) == 0) *entry = id;
          if (id >= 0 && id < a.n_pages) slot = (id << a.page_shift) + (pos & pmask);
        }
      }
      a.positions[row] = pos;
      a.slots[row] = slot;
    }
    __syncthreads();  // the marks are read before the next slice resets them
  }
}

}  // namespace

cudaError_t launch_paged_tables(const TablesArgs& a, cudaStream_t st) {
  constexpr int NT = 512;
  const int grid = std::max(1, std::min(a.rows / NT + (a.rows % NT != 0), 2 * 152));
  const cudaError_t e = launch_dependent(tables_kernel<NT>, dim3(grid), dim3(NT), 0, st, a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tpx
