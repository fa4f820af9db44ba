// k_attn_shared.cu - verification attention of requests that share prefixes: the shared pages are read once a group (sm_103a).
//
// Mathematics: softmax attention over disjoint sets of tokens joins exactly. With scores s_j = q.k_j / sqrt(d) in base 2, a
// set gives m = max s_j, l = sum 2^(s_j - m), o = sum 2^(s_j - m) v_j, and two of them join to m' = max(m1, m2),
// l' = l1 2^(m1 - m') + l2 2^(m2 - m'), o' alike. A query row's tokens are three sets: the prefix that its group shares, the
// rest of its own context, and the tokens of its window up to itself.
//
// The first two are work of the first kernel. Its items are (group, KV head, block of query rows) over the group's prefix,
// where the rows are those of all the group's requests, and (request, KV head, block of rows) over the request's own
// pages; their tiles of 128 tokens, laid end to end, are split evenly over the CTAs. All tokens of an item are
// visible to all its rows, so it needs no mask but the item's end. Each CTA leaves one record (m, l, o) a row of each item
// that it worked on: the item's first CTA at the row's own place, a later one in an area of the CTA's own (a CTA
// can be a later one of at most one item, that which it starts in). The second kernel joins a row's records and
// takes the window's tokens by itself, one warp a row: those are the only tokens that some of a request's rows see and
// others do not.
#include "kap_device.cuh"
#include "kap_launch.h"

#include <algorithm>

namespace kap {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTilePages = 8, kTileTok = kTilePages * kPage;
constexpr int kMaxCtas = 192;      // CTAs of the first kernel at most
constexpr int kMaxBlock = 256;     // rows of an item's block at most
constexpr int kSmemGroups = 1024;  // group offsets kept in shared memory
constexpr int kPlainThreads = 256, kPlainRows = 32;

struct HParams {
  int num_pages, hkv, hq, G, R, max_pages, total_q, num_groups, block;
  const int32_t *bt, *q_offsets, *q_start, *group_off, *prefix_pages;
  const void *K, *V, *q;
  void *out;
  float *lse;
  int64_t *start;   // [num_groups + R + 1] first tile of each entry (a group or a request), and the number of tiles
  float2 *ml[2];    // [total_q][hq] (m, l) of the prefix and of the own context: first CTA's record
  float *o[2];      // [total_q][hq][d]
  float2 *xml;      // [kMaxCtas][block]: later CTAs' records
  float *xo;        // [kMaxCtas][block][d]
  int nb;           // CTAs of the first kernel
  int *err;
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }
__device__ __forceinline__ int row_at(const HParams &p, int r) { return clampi(p.q_offsets[r], 0, p.total_q); }

// A run of tokens and the query rows that see all of them.
struct Entry {
  int q0, rows;       // first query token and number of (token, head in the KV group) rows
  int req;            // the request whose table row names the pages
  int page0, tok0, tok1;  // first page, and the tokens [tok0, tok1) (tok0 = 16 page0)
  int tiles, blocks;  // 128-token tiles; blocks of rows
};

struct Groups {
  const int32_t *off;  // in shared memory where they fit
  // Group of request r, or -1.
  __device__ __forceinline__ int of(const HParams &p, int r) const {
    int lo = 0, hi = p.num_groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (off[mid] <= r) lo = mid; else hi = mid;
    }
    return p.num_groups > 0 && off[lo] <= r && r < off[lo + 1] ? lo : -1;
  }
};

// Shared pages of group g: none where it has fewer than two requests.
__device__ __forceinline__ int shared_pages(const HParams &p, const int32_t *off, int g) {
  const int a = clampi(off[g], 0, p.R), b = clampi(off[g + 1], 0, p.R);
  return b - a < 2 ? 0 : clampi(p.prefix_pages[g], 0, p.max_pages);
}
// Pages that request r takes from its group's item; none when its window starts inside them.
__device__ __forceinline__ int taken_pages(const HParams &p, const Groups &gr, int r) {
  const int g = gr.of(p, r);
  if (g < 0) return 0;
  const int n = shared_pages(p, gr.off, g);
  return n * kPage <= p.q_start[r] ? n : 0;
}

__device__ __forceinline__ Entry entry(const HParams &p, const Groups &gr, int e) {
  Entry x;
  int last;
  if (e < p.num_groups) {
    const int a = clampi(gr.off[e], 0, p.R), b = clampi(gr.off[e + 1], a, p.R);
    x.req = min(a, p.R - 1);
    x.q0 = row_at(p, a);
    last = row_at(p, b);
    x.page0 = 0;
    x.tok1 = shared_pages(p, gr.off, e) * kPage;
  } else {
    x.req = e - p.num_groups;
    x.q0 = row_at(p, x.req);
    last = row_at(p, x.req + 1);
    x.page0 = taken_pages(p, gr, x.req);
    x.tok1 = clampi(p.q_start[x.req], 0, p.max_pages * kPage);
  }
  x.rows = max(last - x.q0, 0) * p.G;
  x.tok0 = x.page0 * kPage;
  x.tiles = x.rows > 0 && x.tok1 > x.tok0 ? (x.tok1 - x.tok0 + kTileTok - 1) / kTileTok : 0;
  x.blocks = (x.rows + p.block - 1) / p.block;
  return x;
}

__device__ __forceinline__ int owner_cta(int64_t x, int64_t E, int nb) {
  return static_cast<int>(((x + 1) * nb - 1) / E);
}

struct Plan {
  int64_t total, begin, end;  // tiles in all, and this CTA's
  int nb;                     // CTAs with tiles
  int entry;                  // the entry that `begin` lies in, and its first tile
  int64_t entry_start;
};

// Every thread of the block takes part; the block has at most 32 warps.
__device__ inline Plan make_plan(const HParams &p, const Groups &gr, int64_t *scratch, int64_t *slot) {
  const int n = p.num_groups + p.R, tid = threadIdx.x, nt = blockDim.x;
  auto count = [&](int e) -> int64_t {
    if (e >= n) return 0;
    const Entry x = entry(p, gr, e);
    return static_cast<int64_t>(x.tiles) * x.blocks * p.hkv;
  };
  const int64_t mine = count(tid);
  int64_t sum = mine;
  for (int e = tid + nt; e < n; e += nt) sum += count(e);
  const int64_t incl = block_inclusive_scan(sum, scratch);
  if (tid == nt - 1) slot[0] = incl;
  __syncthreads();
  Plan pl;
  pl.total = slot[0];
  pl.nb = static_cast<int>(min(pl.total, static_cast<int64_t>(p.nb)));
  pl.begin = pl.end = 0;
  pl.entry = 0;
  pl.entry_start = 0;
  const bool works = static_cast<int>(blockIdx.x) < pl.nb;
  if (works) {
    pl.begin = static_cast<int64_t>(blockIdx.x) * pl.total / pl.nb;
    pl.end = static_cast<int64_t>(blockIdx.x + 1) * pl.total / pl.nb;
  }
  const bool writer = blockIdx.x == 0;
  int64_t base = 0;
  for (int e0 = 0; e0 < n; e0 += nt) {
    const int e = e0 + tid;
    const int64_t c = e0 == 0 ? mine : count(e);
    const int64_t inc = block_inclusive_scan(c, scratch);
    const int64_t first = base + inc - c;
    if (works && first <= pl.begin && pl.begin < first + c) {
      slot[1] = e;
      slot[2] = first;
    }
    if (writer && e < n) p.start[e] = first;
    if (tid == nt - 1) slot[3] = base + inc;
    __syncthreads();
    base = slot[3];
    __syncthreads();
  }
  if (writer && tid == 0) p.start[n] = pl.total;
  if (works) {
    pl.entry = static_cast<int>(slot[1]);
    pl.entry_start = slot[2];
  }
  return pl;
}

__device__ __forceinline__ Groups load_groups(const HParams &p, int32_t *s_off) {
  if (p.num_groups > kSmemGroups) return Groups{p.group_off};
  for (int i = threadIdx.x; i <= p.num_groups; i += blockDim.x) s_off[i] = p.num_groups > 0 ? p.group_off[i] : 0;
  __syncthreads();
  return Groups{s_off};
}

// CTA 0: offsets have to rise from 0 to R.
__device__ __forceinline__ void check_groups(const HParams &p, const Groups &gr) {
  if (blockIdx.x != 0 || p.num_groups == 0) return;
  for (int g = threadIdx.x; g < p.num_groups; g += blockDim.x) {
    const int a = gr.off[g], b = gr.off[g + 1];
    if (a > b || (g == 0 && a != 0) || (g == p.num_groups - 1 && b != p.R)) set_error(p.err, kErrLength);
  }
}

// Where this CTA's record of row n (of the whole item) goes: `later` when an earlier CTA holds the item's first tile.
struct Place {
  float2 *ml;
  float *o;
};
template <int D>
__device__ __forceinline__ Place place(const HParams &p, const Entry &x, int kind, int h, int n, bool later, int cta) {
  if (later) {
    const size_t i = static_cast<size_t>(cta) * p.block + n % p.block;
    return Place{p.xml + i, p.xo + i * D};
  }
  const size_t i = static_cast<size_t>(x.q0 + n / p.G) * p.hq + h * p.G + n % p.G;
  return Place{p.ml[kind] + i, p.o[kind] + i * D};
}

// ------------------------------------------------------------------------------------------------- plain arithmetic
// fp32 pools: a warp takes every eighth row of a block of 32 and all tokens of a tile, a lane every 32nd dim.
template <class T, int D>
__global__ void __launch_bounds__(kPlainThreads) shared_plain_kernel(const HParams p) {
  constexpr int PL = D / 32, RW = kPlainRows / (kPlainThreads / 32);
  __shared__ int32_t s_off[kSmemGroups + 1];
  __shared__ int64_t s_scratch[32], s_slot[4];
  grid_dependency_sync();
  const Groups gr = load_groups(p, s_off);
  check_groups(p, gr);
  const Plan pl = make_plan(p, gr, s_scratch, s_slot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float scale = rsqrtf(static_cast<float>(D)) * kLog2e;
  int e = pl.entry;
  int64_t es = pl.entry_start;
  Entry x{};
  int have = -1;
  for (int64_t at = pl.begin; at < pl.end;) {
    if (have != e) {
      x = entry(p, gr, e);
      have = e;
    }
    const int64_t size = static_cast<int64_t>(x.tiles) * x.blocks * p.hkv;
    if (at >= es + size) {
      es += size;
      ++e;
      continue;
    }
    const int sub = static_cast<int>((at - es) / x.tiles);
    const int t0 = static_cast<int>(at - es - static_cast<int64_t>(sub) * x.tiles);
    const int t1 = static_cast<int>(min(static_cast<int64_t>(x.tiles), t0 + pl.end - at));
    const int h = sub / x.blocks, n0 = (sub - h * x.blocks) * p.block;
    float qv[RW][PL], ov[RW][PL], m[RW], l[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int n = min(n0 + warp + i * (kPlainThreads / 32), x.rows - 1);
      const T *q = static_cast<const T *>(p.q) +
                   (static_cast<size_t>(x.q0 + n / p.G) * p.hq + h * p.G + n % p.G) * D;
#pragma unroll
      for (int k = 0; k < PL; ++k) {
        qv[i][k] = to_f(q[lane + 32 * k]) * scale;
        ov[i][k] = 0.0f;
      }
      m[i] = -INFINITY;
      l[i] = 0.0f;
    }
    const int32_t *bt = p.bt + static_cast<size_t>(x.req) * p.max_pages;
    const int tok_end = min(x.tok1, x.tok0 + t1 * kTileTok);
    for (int tok = x.tok0 + t0 * kTileTok; tok < tok_end; ++tok) {
      const int pg = tok / kPage < p.max_pages ? bt[tok / kPage] : -1;
      if (pg < 0 || pg >= p.num_pages) {
        if (lane == 0) set_error(p.err, kErrPage);
        continue;
      }
      const size_t o = ((static_cast<size_t>(pg) * p.hkv + h) * kPage + tok % kPage) * D + lane;
      const T *kr = static_cast<const T *>(p.K) + o, *vr = static_cast<const T *>(p.V) + o;
      float kv[PL], vv[PL];
#pragma unroll
      for (int k = 0; k < PL; ++k) {
        kv[k] = to_f(kr[32 * k]);
        vv[k] = to_f(vr[32 * k]);
      }
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < PL; ++k) s = fmaf(qv[i][k], kv[k], s);
        s = warp_sum(s);
        const float mn = fmaxf(m[i], s);
        const float a = m[i] == -INFINITY ? 0.0f : exp2f(m[i] - mn), w = s == -INFINITY ? 0.0f : exp2f(s - mn);
        l[i] = l[i] * a + w;
#pragma unroll
        for (int k = 0; k < PL; ++k) ov[i][k] = fmaf(w, vv[k], ov[i][k] * a);
        m[i] = mn;
      }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int n = n0 + warp + i * (kPlainThreads / 32);
      if (n < min(x.rows, n0 + p.block)) {
        const Place pp = place<D>(p, x, e < p.num_groups ? 0 : 1, h, n, t0 > 0, blockIdx.x);
        if (lane == 0) *pp.ml = make_float2(m[i], l[i]);
#pragma unroll
        for (int k = 0; k < PL; ++k) pp.o[lane + 32 * k] = ov[i][k];
      }
    }
    at += t1 - t0;
  }
}

// --------------------------------------------------------------------------------------------- joining the records
// One warp a query row: its records of the prefix and of the own context, and the window's tokens up to itself.
template <class T, int D>
__global__ void __launch_bounds__(128) shared_join_kernel(const HParams p) {
  constexpr int PL = D / 32;  // consecutive dims of a lane
  grid_dependency_sync();
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (wid >= static_cast<int64_t>(p.total_q) * p.hq) return;
  const int t = static_cast<int>(wid / p.hq), hq = static_cast<int>(wid - static_cast<int64_t>(t) * p.hq);
  const int h = hq / p.G;
  int lo = 0, hi = p.R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_offsets[mid] <= t) lo = mid; else hi = mid;
  }
  const int r = lo;
  const Groups gr{p.group_off};
  const int n = p.num_groups + p.R;
  const int64_t total = p.start[n];
  const int nb = static_cast<int>(min(total, static_cast<int64_t>(p.nb)));
  float m = -INFINITY, l = 0.0f, o[PL];
#pragma unroll
  for (int k = 0; k < PL; ++k) o[k] = 0.0f;
  auto join = [&](float2 ml, const float *rec) {
    if (!(ml.y > 0.0f) && ml.x == -INFINITY) return;
    const float mn = fmaxf(m, ml.x);
    const float a = m == -INFINITY ? 0.0f : exp2f(m - mn), b = exp2f(ml.x - mn);
    l = fmaf(l, a, ml.y * b);
#pragma unroll
    for (int k = 0; k < PL; ++k) o[k] = fmaf(rec[lane * PL + k], b, o[k] * a);
    m = mn;
  };
  const bool shares = taken_pages(p, gr, r) > 0;
  for (int kind = 0; kind < 2; ++kind) {
    if (kind == 0 && !shares) continue;
    const int e = kind == 0 ? gr.of(p, r) : p.num_groups + r;
    const Entry x = entry(p, gr, e);
    if (x.tiles == 0) continue;
    const int row = (t - x.q0) * p.G + hq - h * p.G;
    const int64_t first = p.start[e] + (static_cast<int64_t>(h) * x.blocks + row / p.block) * x.tiles;
    const int b0 = owner_cta(first, total, nb), b1 = owner_cta(first + x.tiles - 1, total, nb);
    for (int b = b0; b <= b1; ++b) {
      const Place pp = place<D>(p, x, kind, h, row, b > b0, b);
      join(*pp.ml, pp.o);
    }
  }
  // the window's tokens
  const T *qr = static_cast<const T *>(p.q) + (static_cast<size_t>(t) * p.hq + hq) * D + lane * PL;
  const float scale = rsqrtf(static_cast<float>(D)) * kLog2e;
  float qv[PL];
#pragma unroll
  for (int k = 0; k < PL; ++k) qv[k] = to_f(qr[k]) * scale;
  const int start = p.q_start[r];
  if (start > p.max_pages * kPage && lane == 0) set_error(p.err, kErrPage);   // context past the table's end
  const int pos1 = start > p.max_pages * kPage ? -1 : start + (t - p.q_offsets[r]);
  for (int pos = max(start, 0); pos <= pos1; ++pos) {
    const int pg = pos / kPage < p.max_pages ? p.bt[static_cast<size_t>(r) * p.max_pages + pos / kPage] : -1;
    if (pg < 0 || pg >= p.num_pages) {
      if (lane == 0) set_error(p.err, kErrPage);
      continue;
    }
    const size_t off = ((static_cast<size_t>(pg) * p.hkv + h) * kPage + pos % kPage) * D + lane * PL;
    const T *kr = static_cast<const T *>(p.K) + off, *vr = static_cast<const T *>(p.V) + off;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < PL; ++k) s = fmaf(qv[k], to_f(kr[k]), s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.0f : exp2f(m - mn), w = s == -INFINITY ? 0.0f : exp2f(s - mn);
    l = fmaf(l, a, w);
#pragma unroll
    for (int k = 0; k < PL; ++k) o[k] = fmaf(w, to_f(vr[k]), o[k] * a);
    m = mn;
  }
  T *op = static_cast<T *>(p.out) + (static_cast<size_t>(t) * p.hq + hq) * D + lane * PL;
  const bool none = l == 0.0f && m == -INFINITY;
#pragma unroll
  for (int k = 0; k < PL; ++k) op[k] = from_f<T>(none ? 0.0f : o[k] / l);
  if (lane == 0) p.lse[static_cast<size_t>(t) * p.hq + hq] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

size_t up(size_t b) { return (b + 255) / 256 * 256; }

template <class T, int D> cudaError_t launch_join(const HParams &p, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(p.total_q) * p.hq;
  return launch_pdl(shared_join_kernel<T, D>, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, s, p);
}

}  // namespace

size_t shared_workspace_bytes(int R, int hkv, int hq, int d, int total_q, int num_groups) {
  (void)hkv;
  const size_t rows = static_cast<size_t>(total_q) * hq, extra = static_cast<size_t>(kMaxCtas) * kMaxBlock;
  return up((static_cast<size_t>(num_groups) + R + 1) * 8) + 2 * up(rows * 8) + 2 * up(rows * d * 4) + up(extra * 8) +
         up(extra * d * 4);
}

cudaError_t launch_verify_shared(const PoolArgs &pa, const MapArgs &ma, int total_q, const int32_t *q_offsets,
                                 const int32_t *q_start, int num_groups, const int32_t *group_off,
                                 const int32_t *prefix_pages, const void *q, void *out, float *lse, void *ws, int *err,
                                 cudaStream_t s) {
  HParams p;
  p.num_pages = pa.num_pages;
  p.hkv = pa.hkv;
  p.hq = pa.hq;
  p.G = pa.hq / pa.hkv;
  p.R = ma.R;
  p.max_pages = ma.max_pages;
  p.total_q = total_q;
  p.num_groups = num_groups;
  p.bt = ma.bt;
  p.q_offsets = q_offsets;
  p.q_start = q_start;
  p.group_off = group_off;
  p.prefix_pages = prefix_pages;
  p.K = pa.k;
  p.V = pa.v;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.err = err;
  const size_t rows = static_cast<size_t>(total_q) * pa.hq;
  unsigned char *w = static_cast<unsigned char *>(ws);
  auto take = [&](size_t bytes) {
    unsigned char *at = w;
    w += up(bytes);
    return at;
  };
  p.start = reinterpret_cast<int64_t *>(take((static_cast<size_t>(num_groups) + ma.R + 1) * 8));
  for (int k = 0; k < 2; ++k) p.ml[k] = reinterpret_cast<float2 *>(take(rows * 8));
  for (int k = 0; k < 2; ++k) p.o[k] = reinterpret_cast<float *>(take(rows * pa.d * 4));
  p.xml = reinterpret_cast<float2 *>(take(static_cast<size_t>(kMaxCtas) * kMaxBlock * 8));
  p.xo = reinterpret_cast<float *>(take(static_cast<size_t>(kMaxCtas) * kMaxBlock * pa.d * 4));
  p.nb = std::min(device_sm_count(), kMaxCtas);
  p.block = kPlainRows;
  cudaError_t e;
#define KAP_SHARED(T, D)                                                                                     \
  do {                                                                                                       \
    e = launch_pdl(shared_plain_kernel<T, D>, dim3(p.nb), dim3(kPlainThreads), 0, s, p);                     \
    if (e == cudaSuccess) e = launch_join<T, D>(p, s);                                                       \
  } while (0)
  if (pa.dtype == 0 && pa.d == 128) KAP_SHARED(__nv_bfloat16, 128);
  else if (pa.dtype == 0) KAP_SHARED(__nv_bfloat16, 64);
  else if (pa.d == 128) KAP_SHARED(float, 128);
  else KAP_SHARED(float, 64);
#undef KAP_SHARED
  return e;
}

}  // namespace kap
