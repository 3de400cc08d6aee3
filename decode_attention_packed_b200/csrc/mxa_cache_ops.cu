// The paged cache's bookkeeping kernels: pages and slots for a step's new
// tokens (mxa_extend_tables), and the write of their keys and values
// (mxa_cache_write).
#include <cuda_runtime.h>
#include <stdint.h>

#include "mxa_config.h"
#include "mxa_device.cuh"
#include "mxa_launch.h"

namespace mxa {
namespace {

// ---------------------------------------------------------------------------
// mxa_extend_tables
//
//   have_b = ceil(L_b / P), need_b = ceil((L_b + n_b) / P), take_b = need_b - have_b
//   first_b = sum_{i < b} take_i
//   table[b][have_b + i] = free[first_b + i]              0 <= i < take_b
//   slot[cu_b + t] = table[b][(L_b + t) / P] * P + (L_b + t) % P
//
// A few bytes a row and a token: the call is bound by launch and load
// latency (64 rows of one token, or 8192 tokens of 300 rows: 4.5 us on the
// device, 13 us a call from Python).  One launch: every CTA scans the rows
// itself (chunks of kRows rows in shared memory with a carry, so any number of
// rows works; the offsets and lengths are 8 bytes a row and come from L2) and
// then serves its share of the pages and tokens of the chunk, found by binary
// search.  A page taken in this call is read from the free list, never from
// the table, so no CTA reads what another one writes.
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 256;
constexpr int kRowsPerThread = 4;
constexpr int kRows = kTableThreads * kRowsPerThread;

__global__ void __launch_bounds__(kTableThreads) extend_tables_kernel(const __grid_constant__ TableArgs a) {
  // the chunk's rows: their new tokens [tok0, tok1), the keys held before,
  // the pages that the rows before them take, and the pages they take (-1: refused)
  __shared__ int s_tok0[kRows], s_tok1[kRows], s_len[kRows], s_first[kRows], s_take[kRows];
  __shared__ int s_warp[kTableThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  int carry = 0;  // pages taken by earlier chunks
  int bad = 0;
  const int P = a.page_size;
  const long long capacity = (long long)a.mpps * P;
  int used = 0;  // pages granted, seen by this thread
  for (int b0 = 0; b0 < a.B; b0 += kRows) {
    const int n = min(kRows, a.B - b0);
    // this thread's rows: need, then the scan
    int take[kRowsPerThread], sum = 0;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = tid * kRowsPerThread + i;
      take[i] = 0;
      if (r < n) {
        const int b = b0 + r;
        const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], L0 = a.seqlens[b];
        const int s = min(max(c0, 0), a.total_q), e = min(max(c1, s), a.total_q);
        const int L = L0 < 0 ? 0 : (int)min((long long)L0, capacity);
        if (L != L0) bad |= kErrBadLen;
        if (c1 < c0 || c0 != s || c1 != e || (b == 0 && c0 != 0)) bad |= kErrBadOffsets;
        const int have = (int)(((long long)L + P - 1) / P);
        const long long need = ((long long)L + (e - s) + P - 1) / P;
        const bool wide = need > a.mpps;  // more pages than the row's table holds
        take[i] = wide ? 0 : (int)need - have;
        s_tok0[r] = s;
        s_tok1[r] = e;
        s_len[r] = L;
        s_take[r] = wide ? -1 : take[i];
        sum += take[i];
      }
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int before = carry, total = 0;
#pragma unroll
    for (int w = 0; w < kTableThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    before += incl - sum;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = tid * kRowsPerThread + i;
      if (r < n) {
        s_first[r] = before;
        before += take[i];
        // Rows past the end of the free list take nothing (and keep their length).
        const bool granted = s_take[r] >= 0 && before <= a.num_free;
        if (granted) used = max(used, before);
        if (!granted && s_take[r] != 0) s_take[r] = -1;
        const int b = b0 + r;
        if (b % (int)gridDim.x == (int)blockIdx.x)
          a.new_seqlens[b] = s_len[r] + (s_take[r] >= 0 ? s_tok1[r] - s_tok0[r] : 0);
      }
    }
    __syncthreads();
    const int stride = gridDim.x * kTableThreads;
    // the chunk's pages: free-list entries carry .. carry + total - 1
    const int page_end = min(carry + total, a.num_free);
    for (int i = carry + blockIdx.x * kTableThreads + tid; i < page_end; i += stride) {
      int lo = 0, hi = n - 1;  // last row whose first page is <= i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_first[mid] <= i) lo = mid; else hi = mid - 1;
      }
      const int k = i - s_first[lo];
      if (k < s_take[lo]) {
        const int page = a.free_pages[i], have = (s_len[lo] + P - 1) / P;
        if (page < 0 || page >= a.num_pages) bad |= kErrBadPage;
        a.block_table[(size_t)(b0 + lo) * a.mpps + have + k] = page;
      }
    }
    // the chunk's tokens
    const int tok_begin = s_tok0[0], tok_end = s_tok1[n - 1];
    for (int t = tok_begin + blockIdx.x * kTableThreads + tid; t < tok_end; t += stride) {
      int lo = 0, hi = n - 1;  // last row that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tok0[mid] <= t) lo = mid; else hi = mid - 1;
      }
      int slot = -1;
      if (t >= s_tok0[lo] && t < s_tok1[lo] && s_take[lo] >= 0) {
        const int pos = s_len[lo] + (t - s_tok0[lo]);
        const int p = pos / P, have = (s_len[lo] + P - 1) / P;
        const int page = p < have ? a.block_table[(size_t)(b0 + lo) * a.mpps + p]
                                  : a.free_pages[s_first[lo] + (p - have)];
        if (page >= 0 && page < a.num_pages) slot = page * P + pos % P;
        else bad |= kErrBadPage;
      }
      a.slots[t] = slot;
    }
    carry += total;
    __syncthreads();  // the next chunk's rows replace these
  }
  if (a.B > 0) {  // tokens behind the last row: padding without slots
    const int end = min(max(a.cu_q[a.B], 0), a.total_q);
    for (int t = end + blockIdx.x * kTableThreads + tid; t < a.total_q; t += gridDim.x * kTableThreads) a.slots[t] = -1;
  }
  if (blockIdx.x == 0) {
    // the granted rows' totals rise, so the largest is the number of pages taken
    used = __reduce_max_sync(0xffffffffu, used);
    if (lane == 0) s_warp[warp] = used;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 0; w < kTableThreads / 32; ++w) used = max(used, s_warp[w]);
      *a.pages_used = used;
    }
  }
  if (bad) atomicOr(a.err, bad);
}

// ---------------------------------------------------------------------------
// mxa_cache_write: cache[slot[t]] = new[t] for K and V
//
// Bound by HBM: every key and value is read once and written once.  A
// token's heads are contiguous on both sides (Hkv * D 16-bit values), so one
// warp copies one token's keys or values in 16-byte pieces, four loads in
// flight a lane (16384 tokens of 8 heads of 128: 134 MB read and written in
// 23 us, 5.8 TB/s).
// ---------------------------------------------------------------------------
constexpr int kWriteThreads = 256;

__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const __grid_constant__ WriteArgs a) {
  const int lane = threadIdx.x & 31;
  const long long w0 = (long long)blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5);
  const long long nw = (long long)gridDim.x * (kWriteThreads / 32);
  const int C = a.chunks;  // 16-byte pieces of a token's keys
  grid_launch_dependents();
  grid_dependency_wait();
  int bad = 0;
  for (long long w = w0; w < 2LL * a.total; w += nw) {
    const int t = (int)(w >> 1);
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.pool_tokens) {  // -1: a padded token without a slot
      if (slot != -1) bad = kErrBadPage;
      continue;
    }
    const uint4 *src = (w & 1) ? a.v_new + t * a.v_stride : a.k_new + t * a.k_stride;
    uint4 *dst = ((w & 1) ? a.v_cache : a.k_cache) + (size_t)slot * C;
    int c = lane;
    for (; c + 96 < C; c += 128) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __ldcs(src + c + 32 * i);
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[c + 32 * i] = v[i];
    }
    for (; c < C; c += 32) dst[c] = __ldcs(src + c);
  }
  if (bad && lane == 0) atomicOr(a.err, bad);
}

template <class Args, class Kernel>
mxa_status_t launch_simple(Kernel kernel, const Args &a, int grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return MXA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MXA_OK : MXA_ERR_CUDA;
}

}  // namespace

mxa_status_t launch_extend_tables(TableArgs a, cudaStream_t stream) {
  int sms = 0;
  mxa_status_t st = current_sm_count(&sms);
  if (st == MXA_OK) st = device_error_word(&a.err);
  if (st != MXA_OK) return st;
  // two tokens or rows a thread, at most one CTA per SM: more CTAs only repeat the scan
  const int work = a.total_q > a.B ? a.total_q : a.B;
  const int want = (work + 2 * kTableThreads - 1) / (2 * kTableThreads);
  return launch_simple(extend_tables_kernel, a, want < 1 ? 1 : want < sms ? want : sms, kTableThreads, stream);
}

mxa_status_t launch_cache_write(WriteArgs a, cudaStream_t stream) {
  int sms = 0;
  mxa_status_t st = current_sm_count(&sms);
  if (st == MXA_OK) st = device_error_word(&a.err);
  if (st != MXA_OK) return st;
  const long long warps = 2LL * a.total;
  const long long want = (warps + kWriteThreads / 32 - 1) / (kWriteThreads / 32);
  const long long wave = 8LL * sms;  // resident CTAs of 256 threads
  return launch_simple(cache_write_kernel, a, (int)(want < wave ? want : wave), kWriteThreads, stream);
}

}  // namespace mxa
