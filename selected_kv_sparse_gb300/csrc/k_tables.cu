// k_tables.cu - block tables and slot maps from request lengths, and the return of released pages (sm_103a).
//
// With need[r] = ceil((len[r] + new[r]) / 16) - ceil(len[r] / 16) and E, O the exclusive sums of need and new over the
// requests, request r is granted when E[r] + need[r] <= free_count (or need[r] = 0); its k-th new page is
// free[free_count - 1 - E[r] - k], and its tokens are O[r] .. O[r] + new[r] - 1. Needs of requests that are not granted
// stay in the sum: service is in order, and the sums are one scan.
//
// Bound by latency: 32 decoding requests move about a kilobyte, so what counts is one launch with few dependent loads.
// Every CTA scans all requests itself (tiles of kTile, sums in 64 bits) and keeps the tile's sums in shared memory;
// the tokens and the new pages of the tile are then dealt out over the whole grid in stripes, each found again by a
// binary search in the tile's sums. Long prompts and single tokens are thus spread evenly, no CTA waits for another
// and no workspace is needed. CTA 0 alone writes what there is once per request. A page that is new in this call is
// taken from the stack directly, so no CTA reads a table entry that another one writes.
// On a GB300 a release and an extension take 9.1 us together for 32 requests of one token, 9.9 us for 1024 with long
// prompts among them.
#include "kap_launch.h"
#include "kap_device.cuh"

#include <algorithm>

namespace kap {
namespace {

constexpr int kTabThreads = 512;
constexpr int kPer = 4;                       // requests of a thread per tile
constexpr int kTile = kTabThreads * kPer;

__device__ __forceinline__ int clamp_count(int c, int cap, int *err) {
  if (c < 0 || c > cap) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_error(err, c < 0 ? kErrLength : kErrCapacity);
    return c < 0 ? 0 : cap;
  }
  return c;
}

// Exclusive sums of v[0..kPer) over the block, `total` its sum. Ends with a barrier.
__device__ __forceinline__ void tile_scan(const int64_t *v, int64_t *excl, int64_t &total, int64_t *scratch,
                                          int64_t *s_total) {
  int64_t sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) sum += v[k];
  const int64_t incl = block_inclusive_scan<int64_t>(sum, scratch);
  if (threadIdx.x == kTabThreads - 1) *s_total = incl;
  __syncthreads();
  total = *s_total;
  int64_t at = incl - sum;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    excl[k] = at;
    at += v[k];
  }
}

// Last i < n with a[i] <= x (a ascends, a[0] <= x).
__device__ __forceinline__ int find_last(const int64_t *a, int n, int64_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// First index >= from that belongs to this CTA's stripes of kTabThreads consecutive indices, plus the thread.
__device__ __forceinline__ int64_t stripe_start(int64_t from) {
  const int64_t s = from / kTabThreads;
  const int64_t g = gridDim.x;
  int64_t mine = s - s % g + blockIdx.x;
  if (mine < s) mine += g;
  return mine * kTabThreads + threadIdx.x;
}

__global__ void __launch_bounds__(kTabThreads) extend_kernel(
    int R, int max_pages, int32_t *__restrict__ bt, const int32_t *__restrict__ seq_len,
    const int32_t *__restrict__ new_tokens, const int32_t *__restrict__ free_pages, int free_cap,
    const int32_t *__restrict__ free_count, int32_t *__restrict__ free_count_out, int32_t *__restrict__ tok_offsets,
    int64_t *__restrict__ slot_out, int32_t *__restrict__ pos_out, int max_tokens, int32_t *__restrict__ seq_len_out,
    int32_t *__restrict__ granted_out, int *err) {
  __shared__ int64_t s_tok[kTile], s_page[kTile];  // exclusive sums of new tokens and of needed pages
  __shared__ int32_t s_len[kTile];                 // tokens held, or ~tokens when not granted
  __shared__ int64_t s_scr[kTabThreads / 32], s_total;
  __shared__ int s_taken;
  grid_dependency_sync();
  const int fc = clamp_count(free_count[0], free_cap, err);
  if (threadIdx.x == 0) s_taken = 0;
  int64_t tok0 = 0, page0 = 0;
  for (int base = 0; base < R; base += kTile) {
    const int r0 = base + threadIdx.x * kPer;
    int len[kPer], want[kPer];
    int64_t need[kPer], nw[kPer], et[kPer], ep[kPer];
    bool fits[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const bool in = r0 + k < R;
      len[k] = in ? seq_len[r0 + k] : 0;
      want[k] = in ? new_tokens[r0 + k] : 0;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (len[k] < 0 || want[k] < 0) {
        if (blockIdx.x == 0) set_error(err, kErrLength);
        len[k] = max(len[k], 0);
        want[k] = max(want[k], 0);
      }
      nw[k] = want[k];
      const int64_t old = (static_cast<int64_t>(len[k]) + kPage - 1) / kPage;
      const int64_t all = (static_cast<int64_t>(len[k]) + want[k] + kPage - 1) / kPage;
      fits[k] = all <= max_pages;
      if (!fits[k] && blockIdx.x == 0) set_error(err, kErrCapacity);
      need[k] = fits[k] ? all - old : 0;
    }
    int64_t tsum, psum;
    tile_scan(nw, et, tsum, s_scr, &s_total);
    __syncthreads();
    tile_scan(need, ep, psum, s_scr, &s_total);
    int taken = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = threadIdx.x * kPer + k;
      const int64_t e = page0 + ep[k];
      const bool ok = fits[k] && (need[k] == 0 || e + need[k] <= fc);
      s_tok[i] = tok0 + et[k];
      s_page[i] = e;
      s_len[i] = ok ? len[k] : ~len[k];
      if (ok && need[k] > 0) taken = static_cast<int>(e + need[k]);
      if (blockIdx.x == 0 && r0 + k < R) {
        tok_offsets[r0 + k] = static_cast<int32_t>(min(tok0 + et[k], static_cast<int64_t>(0x7fffffff)));
        granted_out[r0 + k] = ok;
        seq_len_out[r0 + k] = ok ? len[k] + want[k] : len[k];
      }
    }
    if (taken) atomicMax(&s_taken, taken);
    __syncthreads();
    const int n = min(kTile, R - base);
    // new table entries: the needed pages page0 .. page0 + psum - 1, as far as the stack goes
    const int64_t pend = min(page0 + psum, static_cast<int64_t>(fc));
    for (int64_t x = stripe_start(page0); x < pend; x += static_cast<int64_t>(gridDim.x) * kTabThreads) {
      if (x < page0) continue;
      const int i = find_last(s_page, n, x);
      if (s_len[i] < 0) continue;
      const int old = static_cast<int>((static_cast<int64_t>(s_len[i]) + kPage - 1) / kPage);
      const int id = free_pages[fc - 1 - x];
      if (id < 0) set_error(err, kErrPage);
      bt[static_cast<size_t>(base + i) * max_pages + old + (x - s_page[i])] = id;
    }
    // tokens tok0 .. tok0 + tsum - 1, as far as the outputs go
    const int64_t tend = min(tok0 + tsum, static_cast<int64_t>(max_tokens));
    for (int64_t x = stripe_start(tok0); x < tend; x += static_cast<int64_t>(gridDim.x) * kTabThreads) {
      if (x < tok0) continue;
      const int i = find_last(s_tok, n, x);
      const bool ok = s_len[i] >= 0;
      const int len0 = ok ? s_len[i] : ~s_len[i];
      const int64_t pos = len0 + (x - s_tok[i]);
      int64_t slot = -1;
      if (ok) {
        const int old = static_cast<int>((static_cast<int64_t>(len0) + kPage - 1) / kPage);
        const int j = static_cast<int>(pos / kPage);
        const int id = j < old ? bt[static_cast<size_t>(base + i) * max_pages + j]
                               : free_pages[fc - 1 - (s_page[i] + (j - old))];
        if (id >= 0) slot = static_cast<int64_t>(id) * kPage + pos % kPage;
      }
      slot_out[x] = slot;
      pos_out[x] = static_cast<int32_t>(min(pos, static_cast<int64_t>(0x7fffffff)));
    }
    tok0 += tsum;
    page0 += psum;
    __syncthreads();  // the tile's sums are overwritten next
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    tok_offsets[R] = static_cast<int32_t>(min(tok0, static_cast<int64_t>(0x7fffffff)));
    free_count_out[0] = fc - s_taken;
    if (tok0 > max_tokens) set_error(err, kErrCapacity);
  }
}

__global__ void __launch_bounds__(kTabThreads) release_kernel(
    int R, int max_pages, const int32_t *__restrict__ bt, const int32_t *__restrict__ seq_len,
    const int32_t *__restrict__ released, int32_t *__restrict__ free_pages, int free_cap,
    const int32_t *__restrict__ free_count, int32_t *__restrict__ free_count_out, int32_t *__restrict__ seq_len_out,
    int *err) {
  __shared__ int64_t s_page[kTile];
  __shared__ int64_t s_scr[kTabThreads / 32], s_total;
  grid_dependency_sync();
  const int fc = clamp_count(free_count[0], free_cap, err);
  int64_t page0 = 0;
  for (int base = 0; base < R; base += kTile) {
    const int r0 = base + threadIdx.x * kPer;
    int len[kPer], gone[kPer];
    int64_t pages[kPer], ep[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const bool in = r0 + k < R;
      len[k] = in ? seq_len[r0 + k] : 0;
      gone[k] = in ? released[r0 + k] : 0;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      int64_t n = (static_cast<int64_t>(max(len[k], 0)) + kPage - 1) / kPage;
      if (len[k] < 0 || (gone[k] && n > max_pages)) {
        if (blockIdx.x == 0) set_error(err, kErrLength);
        n = min(n, static_cast<int64_t>(max_pages));
      }
      pages[k] = gone[k] ? n : 0;
      if (blockIdx.x == 0 && r0 + k < R) seq_len_out[r0 + k] = gone[k] ? 0 : max(len[k], 0);
    }
    int64_t psum;
    tile_scan(pages, ep, psum, s_scr, &s_total);
#pragma unroll
    for (int k = 0; k < kPer; ++k) s_page[threadIdx.x * kPer + k] = page0 + ep[k];
    __syncthreads();
    const int n = min(kTile, R - base);
    const int64_t pend = min(page0 + psum, static_cast<int64_t>(free_cap) - fc);
    for (int64_t x = stripe_start(page0); x < pend; x += static_cast<int64_t>(gridDim.x) * kTabThreads) {
      if (x < page0) continue;
      const int i = find_last(s_page, n, x);
      free_pages[fc + x] = bt[static_cast<size_t>(base + i) * max_pages + (x - s_page[i])];
    }
    page0 += psum;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (fc + page0 > free_cap) set_error(err, kErrCapacity);
    free_count_out[0] = static_cast<int32_t>(min(fc + page0, static_cast<int64_t>(free_cap)));
  }
}

// The same over a pool with packed pages: ids below P16 go to the stack s16, the P4 ids after them to s4. Where an id goes
// depends on the kinds of all before it, so one CTA walks the released entries in order, kTile a turn, and scans both
// kinds at once (a count in either half of a word), and none waits for another. On a GB300 2049 pages take 5.8 us, 16392
// (eight requests) 22 us, 262144 310 us; the release of one kind 4.4, 17 and 24 us.
__global__ void __launch_bounds__(kTabThreads) release_by_kind_kernel(
    int R, int max_pages, const int32_t *__restrict__ bt, const int32_t *__restrict__ seq_len,
    const int32_t *__restrict__ released, int P16, int P4, StackArgs s16, StackArgs s4, int32_t *__restrict__ seq_len_out,
    int *err) {
  __shared__ int64_t s_page[kTile];
  __shared__ int64_t s_scr[kTabThreads / 32], s_total;
  grid_dependency_sync();
  int64_t n16 = clamp_count(s16.count[0], s16.cap, err), n4 = clamp_count(s4.count[0], s4.cap, err);
  for (int base = 0; base < R; base += kTile) {
    const int r0 = base + threadIdx.x * kPer;
    int64_t pages[kPer], ep[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const bool in = r0 + k < R;
      const int len = in ? seq_len[r0 + k] : 0, gone = in ? released[r0 + k] : 0;
      int64_t n = (static_cast<int64_t>(max(len, 0)) + kPage - 1) / kPage;
      if (len < 0 || (gone && n > max_pages)) {
        set_error(err, kErrLength);
        n = min(n, static_cast<int64_t>(max_pages));
      }
      pages[k] = gone ? n : 0;
      if (in) seq_len_out[r0 + k] = gone ? 0 : max(len, 0);
    }
    int64_t psum;
    tile_scan(pages, ep, psum, s_scr, &s_total);
#pragma unroll
    for (int k = 0; k < kPer; ++k) s_page[threadIdx.x * kPer + k] = ep[k];
    __syncthreads();
    const int n = min(kTile, R - base);
    for (int64_t at = 0; at < psum; at += kTile) {
      const int64_t x0 = at + threadIdx.x * kPer;
      int i = x0 < psum ? find_last(s_page, n, x0) : 0;
      int id[kPer];
      int64_t v[kPer], ex[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int64_t x = x0 + k;
        id[k] = -1;
        v[k] = 0;
        if (x < psum) {
          while (i + 1 < n && s_page[i + 1] <= x) ++i;
          id[k] = bt[static_cast<size_t>(base + i) * max_pages + (x - s_page[i])];
          if (id[k] < 0 || id[k] >= P16 + P4) set_error(err, kErrPage);
          else v[k] = id[k] < P16 ? 1 : int64_t(1) << 32;
        }
      }
      int64_t sum;
      tile_scan(v, ex, sum, s_scr, &s_total);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (v[k] == 0) continue;
        const StackArgs &s = v[k] == 1 ? s16 : s4;
        const int64_t to = v[k] == 1 ? n16 + (ex[k] & 0xffffffff) : n4 + (ex[k] >> 32);
        if (to < s.cap) s.ids[to] = id[k];
      }
      n16 += sum & 0xffffffff;
      n4 += sum >> 32;
      __syncthreads();  // the scan's memory is used again
    }
    __syncthreads();  // and the tile's sums
  }
  if (threadIdx.x == 0) {
    if (n16 > s16.cap || n4 > s4.cap) set_error(err, kErrCapacity);
    s16.count_out[0] = static_cast<int32_t>(min(n16, static_cast<int64_t>(s16.cap)));
    s4.count_out[0] = static_cast<int32_t>(min(n4, static_cast<int64_t>(s4.cap)));
  }
}

// CTAs: enough for one stripe a thread each, at most one per SM.
int table_grid(int64_t items) {
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(1, (items + kTabThreads - 1) / kTabThreads),
                                            device_sm_count()));
}

}  // namespace

cudaError_t launch_extend_tables(int R, int max_pages, int32_t *bt, const int32_t *seq_len, const int32_t *new_tokens,
                                 const int32_t *free_pages, int free_cap, const int32_t *free_count,
                                 int32_t *free_count_out, int32_t *tok_offsets, int64_t *slot_out, int32_t *pos_out,
                                 int max_tokens, int32_t *seq_len_out, int32_t *granted_out, int *err,
                                 cudaStream_t s) {
  return launch_pdl(extend_kernel, dim3(table_grid(max_tokens)), dim3(kTabThreads), 0, s, R, max_pages, bt, seq_len,
                    new_tokens, free_pages, free_cap, free_count, free_count_out, tok_offsets, slot_out, pos_out,
                    max_tokens, seq_len_out, granted_out, err);
}

cudaError_t launch_release_tables(int R, int max_pages, const int32_t *bt, const int32_t *seq_len,
                                  const int32_t *released, int32_t *free_pages, int free_cap,
                                  const int32_t *free_count, int32_t *free_count_out, int32_t *seq_len_out, int *err,
                                  cudaStream_t s) {
  return launch_pdl(release_kernel, dim3(table_grid(static_cast<int64_t>(R) * 8)), dim3(kTabThreads), 0, s, R,
                    max_pages, bt, seq_len, released, free_pages, free_cap, free_count, free_count_out, seq_len_out,
                    err);
}

cudaError_t launch_release_by_kind(int R, int max_pages, const int32_t *bt, const int32_t *seq_len,
                                   const int32_t *released, int P16, int P4, const StackArgs &s16, const StackArgs &s4,
                                   int32_t *seq_len_out, int *err, cudaStream_t s) {
  return launch_pdl(release_by_kind_kernel, dim3(1), dim3(kTabThreads), 0, s, R, max_pages, bt, seq_len, released, P16, P4,
                    s16, s4, seq_len_out, err);
}

}  // namespace kap
