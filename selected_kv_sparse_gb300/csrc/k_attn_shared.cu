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
//
// bf16 pools run on tcgen05 (shared_tc_kernel, which says how), fp32 pools in plain arithmetic. In graphs: 32 requests on one
// prefix of 32768 tokens 66 us (pages alone 25, at the measured copy rate), 64 in 5 groups with windows of 5 156 us (54), 8 on
// 131072 with windows of 8 264 us (products alone 90, pages 81); kap_attn_verify over the same tables 522, 564 and 687.
#include "kap_device.cuh"
#include "kap_launch.h"
#include "kap_tma.h"

#include <algorithm>
#include <type_traits>

namespace kap {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTilePages = 8, kTileTok = kTilePages * kPage;
constexpr int kMaxCtas = 192;      // CTAs of the first kernel at most
constexpr int kMaxBlock = 256;     // rows of an item's block at most
constexpr int kSmemGroups = 1024;  // group offsets kept in shared memory
// Lengths on the line that is shared out, about 0.7 us each: a tile under up to 128 rows takes 2 (what its 64 KB take to
// come at an SM's share of the measured copy rate), under more 3 (four products and two softmaxes); starting and ending an
// item takes 4.
constexpr int kTileCost = 2, kWideCost = 3, kItemCost = 4;
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
  // A block's length on the line is its start's and then its tiles'. All blocks but the last are whole.
  __device__ __forceinline__ int cost(const HParams &p, int block) const {
    return p.block > 128 && rows - block * p.block > 128 ? kWideCost : kTileCost;
  }
  __device__ __forceinline__ int64_t span(int w) const { return static_cast<int64_t>(tiles) * w + kItemCost; }
  __device__ __forceinline__ int64_t of_head(const HParams &p) const {
    return tiles == 0 ? 0 : (blocks - 1) * span(cost(p, 0)) + span(cost(p, blocks - 1));
  }
  __device__ __forceinline__ int64_t length(const HParams &p) const { return of_head(p) * p.hkv; }
  // Where the tiles of (head, block) start, from the entry's own start on.
  __device__ __forceinline__ int64_t first_tile(const HParams &p, int h, int block) const {
    return h * of_head(p) + block * span(cost(p, 0)) + kItemCost;
  }
};
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {   // of numbers >= 0; 32 bits where they do
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

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
  return static_cast<int>(quotient((x + 1) * nb - 1, E));
}
// CTAs that take part: every part holds a tile's start at least, so every CTA between an item's first and last has a record.
__device__ __forceinline__ int parts(const HParams &p, int64_t total) {
  return static_cast<int>(max(int64_t(total > 0), min(total / kWideCost, static_cast<int64_t>(p.nb))));
}

// Where a CTA's part of the line starts: an entry, a head and block of it, and units into that block.
struct Plan {
  Entry x;
  int entry, h, block, from;
  int64_t left;        // the part's length
};
struct PlanSlots {
  int64_t total, base;
  Plan plan;
};

// Every thread of the block takes part; the block has at most 32 warps.
__device__ inline Plan make_plan(const HParams &p, const Groups &gr, int64_t *scratch, PlanSlots *slot) {
  const int n = p.num_groups + p.R, tid = threadIdx.x, nt = blockDim.x;
  const bool writer = blockIdx.x == 0;
  Entry x{};
  int64_t c = 0, sum = 0, base = 0, begin = 0, end = 0;
  if (tid == 0) slot->plan.left = 0;
  for (int pass = 0; pass < 2; ++pass) {   // the sum of all lengths; then where each entry starts
    for (int e0 = 0; e0 < n; e0 += nt) {
      const int e = e0 + tid;
      if (pass == 0 || n > nt) {
        c = 0;
        if (e < n) {
          x = entry(p, gr, e);
          c = x.length(p);
        }
      }
      if (pass == 0) {
        sum += c;
        continue;
      }
      const int64_t incl = block_inclusive_scan(c, scratch), first = base + incl - c;
      if (first <= begin && begin < first + c && begin < end) {
        const int64_t in = begin - first, per_head = x.of_head(p), whole = x.span(x.cost(p, 0));
        Plan pl;
        pl.x = x;
        pl.entry = e;
        pl.h = static_cast<int>(quotient(in, per_head));
        const int64_t in_head = in - pl.h * per_head;
        pl.block = min(static_cast<int>(quotient(in_head, whole)), x.blocks - 1);
        pl.from = static_cast<int>(in_head - pl.block * whole);
        pl.left = end - begin;
        slot->plan = pl;
      }
      if (writer && e < n) p.start[e] = first;
      if (tid == nt - 1) slot->base = base + incl;
      __syncthreads();
      base = slot->base;
      __syncthreads();
    }
    if (pass == 0) {
      const int64_t incl = block_inclusive_scan(sum, scratch);
      if (tid == nt - 1) slot->total = incl;
      __syncthreads();
      const int64_t total = slot->total;
      const int nb = parts(p, total), cta = static_cast<int>(blockIdx.x);
      if (cta < nb) {
        begin = quotient(cta * total, nb);
        end = quotient((cta + 1) * total, nb);
      }
      if (writer && tid == 0) p.start[n] = total;
    }
  }
  return slot->plan;
}

__device__ __forceinline__ Groups load_groups(const HParams &p, int32_t *s_off) {
  if (p.num_groups > kSmemGroups) return Groups{p.group_off};
  for (int i = threadIdx.x; i <= p.num_groups; i += blockDim.x) s_off[i] = p.num_groups > 0 ? p.group_off[i] : 0;
  __syncthreads();
  return Groups{s_off};
}

// CTA 0: a group's offsets have to rise from 0 to R, those of the windows within [0, total_q].
__device__ __forceinline__ void check_offsets(const HParams &p, const Groups &gr) {
  if (blockIdx.x != 0) return;
  for (int r = threadIdx.x; r < p.R; r += blockDim.x) {
    const int a = p.q_offsets[r], b = p.q_offsets[r + 1];
    if (a < 0 || a > b || b > p.total_q) set_error(p.err, kErrLength);
  }
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

// The segments of a CTA's part, in order: runs of tiles of one (item, block of rows).
struct Segment {
  Entry x;
  int e, h, n0, rows, t0, n;  // tiles [t0, t0 + n) of the block's
};
struct Walker {
  const HParams &p;
  const Groups gr;
  Plan w;
  __device__ __forceinline__ Walker(const HParams &p_, const Plan &pl) : p(p_), gr{p_.group_off}, w(pl) {}
  __device__ __forceinline__ bool next(Segment &s) {
    while (w.left > 0) {
      if (w.x.tiles == 0) {
        if (++w.entry >= p.num_groups + p.R) return false;
        w.x = entry(p, gr, w.entry);
        continue;
      }
      const int cost = w.x.cost(p, w.block), span = static_cast<int>(w.x.span(cost));
      const int to = static_cast<int>(min(static_cast<int64_t>(span), w.from + w.left));
      auto tiles_before = [&](int at) {   // tiles that start before unit `at`
        const int u = max(at - kItemCost, 0) + cost - 1;
        return cost == 2 ? u >> 1 : u / 3;
      };
      s.t0 = tiles_before(w.from);
      s.n = tiles_before(to) - s.t0;
      s.x = w.x;
      s.e = w.entry;
      s.h = w.h;
      s.n0 = w.block * p.block;
      s.rows = min(w.x.rows - s.n0, p.block);
      w.left -= to - w.from;
      w.from = 0;
      if (++w.block == w.x.blocks) {
        w.block = 0;
        if (++w.h == p.hkv) {
          w.h = 0;
          w.x.tiles = 0;   // on to the next entry
        }
      }
      if (s.n > 0) return true;   // else no more than the item's start, or the rest of a tile
    }
    return false;
  }
};
static_assert(kTileCost == 2 && kWideCost == 3, "Walker divides by these");

// ------------------------------------------------------------------------------------------------- plain arithmetic
// fp32 pools: a warp takes every eighth row of a block of 32 and all tokens of a tile, a lane every 32nd dim.
template <class T, int D>
__global__ void __launch_bounds__(kPlainThreads) shared_plain_kernel(const HParams p) {
  constexpr int PL = D / 32, RW = kPlainRows / (kPlainThreads / 32);
  __shared__ int32_t s_off[kSmemGroups + 1];
  __shared__ int64_t s_scratch[32];
  __shared__ PlanSlots s_slot;
  grid_dependency_sync();
  const Groups gr = load_groups(p, s_off);
  check_offsets(p, gr);
  const Plan pl = make_plan(p, gr, s_scratch, &s_slot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float scale = rsqrtf(static_cast<float>(D)) * kLog2e;
  Walker walk(p, pl);
  Segment sg;
  while (walk.next(sg)) {
    const Entry &x = sg.x;
    const int h = sg.h, n0 = sg.n0, t0 = sg.t0, t1 = sg.t0 + sg.n;
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
        const Place pp = place<D>(p, x, sg.e < p.num_groups ? 0 : 1, h, n, t0 > 0, blockIdx.x);
        if (lane == 0) *pp.ml = make_float2(m[i], l[i]);
#pragma unroll
        for (int k = 0; k < PL; ++k) pp.o[lane + 32 * k] = ov[i][k];
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------- tensor cores
// bf16 pools. S[128 rows x 128 tokens] = Q . K^T (tcgen05.mma, M = 128, both operands K-major in shared memory), softmax with
// a thread a row, P back into the tensor memory that S had, as bf16, O[128 rows x d] += P . V (A from tensor memory, V read
// MN-major from shared memory). Two streams of softmax warps, each with an S and an O, take turns at the tensor core:
// an item's block of up to 128 rows gives its even tiles to one and its odd tiles to the other and joins the two at the
// end; a block of up to 256 rows gives each stream 128 of them, and both read every tile.
// P is rounded to bf16 (2^-8 of a weight at most), since a product takes both operands in one 16-bit type; its sum l is of
// the unrounded weights, in fp32. kap_attn_verify does the same at d 128; at d 64 it keeps P in fp32, in a plain kernel that
// takes 28 ms where this one takes 54 us (32 requests on 32768 tokens).
// Warps: 0-3 and 4-7 the streams' softmax (thread = row; they also bring the first segment's queries), 8 and 9 the pages,
// four of each tile, 8 the tile records, 10 the tcgen05 issuer, 11 the later segments' queries. A page of a head is one TMA
// request (about 50 ns of its issuing warp each).
// In shared memory 8 rows of 64 columns are one swizzled block of 1 KB; a K or V tile holds, for each group of 8
// tokens, the blocks of its d / 64 column halves. K and V tiles share a ring.
// A barrier's parity tells a phase from its neighbours only to a thread that has seen every phase before it, so the page
// warps and the issuer watch the ring's places in order and miss none. Every wait is bounded, and no role waits on a
// block-wide barrier.
constexpr int kTcThreads = 384;
constexpr int kTcBlock = 256;
constexpr float kRescale = 8.0f;  // log2: the reference of a row's weights follows its maximum when 2^8 behind

// A tile's record, 32 bytes: tiles of 128 dims leave little shared memory beside the ring.
struct TileInfo {
  int flags, idx, n, tp;   // tile idx of the segment's n; tp: tokens, and from bit 8 on which of its pages are in the pool
  int h, n0, rows, q0;     // rows of the block, from row n0 of the item on
};
constexpr int kValid = 1, kFirst = 2, kLast = 4, kTwo = 8, kQbuf = 16, kKind = 32, kLater = 64;
constexpr int kQuse = 8;  // from this bit on, 2 bits each: how often the two query buffers were filled before, modulo 4

template <int D>
struct Tc {
  static constexpr int ATOM = 128 * 128;               // 64 columns of 128 query rows
  static constexpr int GROUP = 16 * D;                 // 8 tokens of a K or V tile
  static constexpr int UNIT = 128 * D * 2;             // a K or V tile, or 128 query rows
  static constexpr int NU = D == 128 ? 5 : 10;         // ring of tiles
  static constexpr int kMeta = D == 128 ? 4 : 8;       // tile records in flight
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_Q = NU * UNIT;
  static constexpr int OFF_INFO = OFF_Q + 2 * UNIT;
  static constexpr int OFF_X = OFF_INFO + kMeta * static_cast<int>(sizeof(TileInfo));  // m [2][128], l of stream 1 [128]
  // full, empty [NU]; mfull, mfree [kMeta]; qfull, qempty, sfull, pfull, ofull [2]; xready, xdone, drain
  static constexpr int NBAR = 2 * NU + 2 * kMeta + 10 + 3;
  static constexpr int OFF_BAR = OFF_X + 3 * 128 * 4;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;  // the tensor memory's address and the abort flag
  static constexpr int ALLOC = OFF_TMEM + 16;          // leaves the SM 1 KB: a CTA of the joining kernel fits beside
  static_assert(ALLOC <= 226 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ float fast_exp2(float x) {  // relative error about 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The issuing warp stays together and one elected lane acts: descriptors then live in uniform registers, and a product
// takes 15 to 20 cycles to issue where a branch for one lane takes 52 (128 x 128 x 16 itself takes 64).
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p;
}
// D[tmem] (+)= A[smem] * B[smem], bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void umma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem].
__device__ __forceinline__ void umma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_by(uint32_t lead, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
// One page of a head through the 4-D map of make_page_map: 2 groups of 8 tokens, with their column halves.
__device__ __forceinline__ void tma_load_4d(void *dst_smem, const void *tmap, int group, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], [%4];" ::
          "r"(smem_u32(dst_smem)),
      "l"(tmap), "r"(0), "r"(group), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void store32(float *p, const float *v) {   // 32 bytes, on a multiple of 32
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void touch(const int32_t *p) {
  asm volatile("{\n\t.reg .b32 v;\n\tld.global.ca.b32 v, [%0];\n\t}" ::"l"(p));
}
__device__ __forceinline__ void mbar_arrive8(uint64_t *bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], 8;" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A block's query rows [first, first + rows) into a buffer of 128, by threads i of n. Not waited for.
template <int D>
__device__ __forceinline__ void load_queries(const HParams &p, const Segment &s, int first, int rows, unsigned char *dst,
                                             int i, int n) {
  constexpr int CH = D / 8;   // 16-byte pieces of a row
  const __nv_bfloat16 *qg = static_cast<const __nv_bfloat16 *>(p.q);
  for (int c = i; c < rows * CH; c += n) {
    const int row = c / CH, k = c % CH, r = s.n0 + first + row;
    const int t = r / p.G, g = r - t * p.G;
    cp_async16(dst + (k >> 3) * Tc<D>::ATOM + (row >> 3) * 1024 + (row & 7) * 128 + (((k & 7) ^ (row & 7)) << 4),
               qg + (static_cast<size_t>(s.x.q0 + t) * p.hq + s.h * p.G + g) * D + k * 8);
  }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    shared_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const HParams p) {
  using L = Tc<D>;
  constexpr int NU = L::NU, kMeta = L::kMeta;
  // The only shared memory of the kernel, so its base is where the SM's own first KB ends.
  extern __shared__ __align__(1024) unsigned char sm[];
  if (smem_u32(sm) & 1023u) {
    if (threadIdx.x == 0) set_error(p.err, kErrTimeout);
    return;
  }
  unsigned char *ring = sm + L::OFF_RING, *Qs = sm + L::OFF_Q;
  TileInfo *info = reinterpret_cast<TileInfo *>(sm + L::OFF_INFO);
  float *xm = reinterpret_cast<float *>(sm + L::OFF_X);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::OFF_BAR);
  uint64_t *full = bars, *empty = full + NU, *mfull = empty + NU, *mfree = mfull + kMeta, *qfull = mfree + kMeta;
  uint64_t *qempty = qfull + 2, *sfull = qempty + 2, *pfull = sfull + 2, *ofull = pfull + 2, *xready = ofull + 2;
  uint64_t *xdone = xready + 1, *drain = xready + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::OFF_TMEM);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < L::NBAR; ++i) mbar_init(&bars[i], 1);
    for (int i = 0; i < kMeta; ++i) mbar_init(&mfree[i], 9);  // 8 softmax warps and the issuer
    for (int i = 0; i < NU; ++i) mbar_init(&full[i], 2);  // the two page warps
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], 8);
      mbar_init(&qempty[i], 2);
      mbar_init(&pfull[i], 4);
    }
    mbar_init(xready, 8);
    mbar_init(xdone, 8);
    fence_barrier_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_sync();

  // what the plan reads is asked for at once; its own loads then find it near
  for (int i = tid; i <= p.R; i += kTcThreads) {
    touch(p.q_offsets + i);
    if (i < p.R) touch(p.q_start + i);
  }
  for (int i = tid; i < p.num_groups; i += kTcThreads) touch(p.prefix_pages + i);
  // the plan's scratch lies where the ring will be
  const Groups gs = load_groups(p, reinterpret_cast<int32_t *>(ring + 512));
  check_offsets(p, gs);
  const Plan pl = make_plan(p, gs, reinterpret_cast<int64_t *>(ring), reinterpret_cast<PlanSlots *>(ring + 256));
  fence_proxy_async_smem();
  __syncthreads();
  const uint32_t tmem = *tmem_slot;   // S of stream s at column 128 s, O at 256 + 128 s

  auto wait = [&](uint64_t *bar, int phase) -> bool {   // the whole warp
    const bool ok = *abort_flag == 0 && mbar_wait(bar, phase & 1, p.err);
    if (__all_sync(0xffffffffu, ok)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp == 8 || warp == 9) {
    // ------------------------------------------------------------------------------------------------- pages
    const int part = (warp - 8) * (kTilePages / 2);   // this warp's pages of a tile: part .. part + 3
    Walker walk(p, pl);
    Segment s{};
    int u = 0, i = 0, seg = 0, uses[2] = {0, 0}, qflags = 0, freed = 0, issued = 0;
    int page = -1;
    bool more = walk.next(s);
    auto fetch = [&]() {   // page lane of tile i of the segment
      const int j = s.x.page0 + (s.t0 + i) * kTilePages + lane;
      page = lane < kTilePages && j < p.max_pages && j * kPage < s.x.tok1
                 ? p.bt[static_cast<size_t>(s.x.req) * p.max_pages + j] : -1;
    };
    if (more) fetch();
    bool stop = false;
    for (; !stop; ++u) {
      const int mi = u % kMeta;
      if (part == 0 && u >= kMeta && !wait(&mfree[mi], u / kMeta - 1)) break;
      if (!more) {
        if (part == 0 && lane == 0) {
          info[mi].flags = 0;
          mbar_arrive(&mfull[mi]);
        }
        break;
      }
      const int tok = s.x.tok0 + (s.t0 + i) * kTileTok, ntok = min(kTileTok, s.x.tok1 - tok);
      const int npg = (ntok + kPage - 1) / kPage;
      const bool in = lane < npg, ok = in && page >= 0 && page < p.num_pages;
      if (in && !ok) set_error(p.err, kErrPage);
      const uint32_t pages = __ballot_sync(0xffffffffu, ok);
      const int group0 = (page * p.hkv + s.h) * (kPage / 8);
      if (part == 0) {
        if (i == 0) {   // a new segment: its query buffers
          const bool two = s.rows > 128;
          const int qbuf = two ? 0 : (seg & 1);
          qflags = (two ? kTwo : 0) | (qbuf ? kQbuf : 0) | ((uses[0] & 3) << kQuse) | ((uses[1] & 3) << (kQuse + 2)) |
                   (s.e < p.num_groups ? 0 : kKind) | (s.t0 > 0 ? kLater : 0);
          if (two || qbuf == 0) ++uses[0];
          if (two || qbuf == 1) ++uses[1];
          ++seg;
        }
        if (lane == 0) {
          info[mi] = TileInfo{kValid | qflags | (i == 0 ? kFirst : 0) | (i == s.n - 1 ? kLast : 0), i, s.n,
                              ntok | (static_cast<int>(pages) << 8), s.h, s.n0, s.rows, s.x.q0};
          mbar_arrive(&mfull[mi]);
        }
      }
      const uint32_t mine = (pages >> part) & 0xf;
#pragma unroll 1
      for (int v = 0; v < 2 && !stop; ++v) {   // keys, then values
        const int un = 2 * u + v, st = un % NU;
        while (freed <= un - NU && wait(&empty[freed % NU], freed / NU)) ++freed;
        if (freed <= un - NU) {
          stop = true;
          break;
        }
        unsigned char *dst = ring + st * L::UNIT;
        if (v == 1 && mine != 0xf) {   // values that no copy brings must be finite: their weights are zero
          for (int j = part; j < part + 4; ++j)
            if (!((pages >> j) & 1))
              for (int c = lane; c < kPage * D / 8; c += 32)
                *reinterpret_cast<uint4 *>(dst + j * 2 * L::GROUP + c * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[st], __popc(mine) * kPage * D * 2);
        __syncwarp();
        if (ok && (lane & ~3) == part) tma_load_4d(dst + lane * 2 * L::GROUP, v == 0 ? &tmK : &tmV, group0, &full[st]);
        issued = un + 1;
      }
      if (stop) break;
      if (++i == s.n) {
        more = walk.next(s);
        i = 0;
      }
      if (more) fetch();
    }
    // after an abort, copies in flight are waited for (bounded) before the CTA leaves
    if (*abort_flag)
      for (int un = max(0, issued - NU); un < issued; ++un) mbar_wait(&full[un % NU], (un / NU) & 1, nullptr);
  } else if (warp == 11) {
    // ----------------------------------------------------------------------------------------------- queries
    Walker walk(p, pl);
    Segment s;
    int uses[2] = {0, 0};
    bool stop = false;
    for (int seg = 0; !stop && walk.next(s); ++seg) {
      const bool two = s.rows > 128;
      for (int b = 0; b < 2; ++b) {
        if (!two && b != (seg & 1)) continue;
        if (seg > 0) {
          if (uses[b] > 0 && !wait(&qempty[b], uses[b] - 1)) {
            stop = true;
            break;
          }
          const int first = two ? 128 * b : 0;
          load_queries<D>(p, s, first, min(s.rows - first, 128), Qs + b * L::UNIT, lane, 32);
        }
        ++uses[b];
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (seg > 0 && !stop) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (two || (seg & 1) == 0) mbar_arrive8(&qfull[0]);
          if (two || (seg & 1) == 1) mbar_arrive8(&qfull[1]);
        }
      }
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------------------------------------------- issuer
    // Whichever stream has its operands: P . V once P is written and, right behind it, S of the stream's next tile (they
    // share tensor memory, and what one thread issues is carried out in order). So the streams fall out of step, and one's
    // products run under the other's softmax.
    {
      const uint32_t lead = elect_lane();
      auto test = [&](uint64_t *bar, int phase) { return __all_sync(0xffffffffu, mbar_test(bar, phase & 1)) != 0; };
      // A stream: `cur` is the tile whose S is issued and whose P . V is not (busy), `next` the one after it (known).
      int tn[2] = {0, 0}, tc[2] = {-1, -1}, done[2] = {0, 0}, released = 0;
      bool busy[2] = {false, false}, known[2] = {false, false}, over[2] = {false, false};
      int landed = 0, qseen[2] = {0, 0};   // units of the ring and fillings of the query buffers seen
      TileInfo cur[2], next[2];
      const uint32_t idesc_s = idesc_bf16(128, 128, 0, 0), idesc_o = idesc_bf16(128, D, 0, 1);
      auto has_landed = [&](int un) {
        while (landed <= un && test(&full[landed % NU], landed / NU)) ++landed;
        return landed > un;
      };
      uint32_t idle = 0;
      while (true) {
        bool progressed = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int o = 1 - s;
          if (!known[s] && !over[s] && test(&mfull[tn[s] % kMeta], tn[s] / kMeta)) {
            next[s] = info[tn[s] % kMeta];
            progressed = true;
            if (!(next[s].flags & kValid)) over[s] = true;
            else if ((next[s].flags & kTwo) || (next[s].idx & 1) == s) known[s] = true;
            else ++tn[s];   // the other stream's
          }
          bool gave_v = false, gave_k = false, last = false;
          int vu = 0;
          if (busy[s]) {
            vu = 2 * tc[s] + 1;
            if (!has_landed(vu) || !test(&pfull[s], done[s])) continue;
            tc_fence_after();
            const bool two = (cur[s].flags & kTwo) != 0;
            const uint64_t vd = smem_desc(smem_u32(ring + (vu % NU) * L::UNIT), 1024, L::GROUP, 2);
            const bool fresh = two ? cur[s].idx == 0 : cur[s].idx < 2;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ts(lead, tmem + 256 + 128 * s, tmem + 128 * s + kk * 8, vd + (kk * 2 * L::GROUP >> 4), idesc_o,
                           (kk > 0 || !fresh) ? 1u : 0u);
            // who uses a tile last gives it back
            gave_v = !two || tc[o] > tc[s] || (tc[o] == tc[s] && !busy[o]);
            last = two ? (cur[s].flags & kLast) != 0 : cur[s].idx + 2 >= cur[s].n;
            if (last) commit_by(lead, &ofull[s]);
            ++done[s];
            busy[s] = false;
            progressed = true;
          }
          int ku = 0;
          if (known[s]) {
            const TileInfo &m = next[s];
            const bool two = (m.flags & kTwo) != 0;
            const int b = two ? s : ((m.flags & kQbuf) ? 1 : 0);
            ku = 2 * tn[s];
            bool ready = has_landed(ku);
            if (ready && (two ? m.idx == 0 : m.idx < 2)) {   // the stream's first use of its queries
              while (test(&qfull[b], b ? qseen[1] : qseen[0])) b ? ++qseen[1] : ++qseen[0];
              ready = (((b ? qseen[1] : qseen[0]) - (m.flags >> (kQuse + 2 * b))) & 3) == 1;
            }
            if (ready) {
              tc_fence_after();
              // a descriptor counts its address in 16 bytes, and no sum here carries out of that field
              const uint64_t qd = smem_desc(smem_u32(Qs + b * L::UNIT), 16, 1024, 2);
              const uint64_t kd = smem_desc(smem_u32(ring + (ku % NU) * L::UNIT), 16, L::GROUP, 2);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_ss(lead, tmem + 128 * s, qd + (((kk >> 2) * L::ATOM + (kk & 3) * 32) >> 4),
                          kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
              commit_by(lead, &sfull[s]);
              gave_k = !two || tn[o] > tn[s];
              if (two ? (m.flags & kLast) != 0 : m.idx + 2 >= m.n) {   // its last use of them; a buffer counts two
                commit_by(lead, &qempty[b]);
                if (two || m.n == 1) commit_by(lead, &qempty[b]);
              }
              cur[s] = m;
              tc[s] = tn[s]++;
              busy[s] = true;
              known[s] = false;
              progressed = true;
            }
          }
          if (gave_v) commit_by(lead, &empty[vu % NU]);
          if (gave_k) commit_by(lead, &empty[ku % NU]);
        }
        if (over[0] && over[1] && !busy[0] && !busy[1]) break;
        const int passed = min(tn[0], tn[1]);   // both streams know what they need of the tiles before
        if (released < passed) {
          __syncwarp();   // every lane has read them
          for (; released < passed; ++released)
            if (lane == 0) mbar_arrive(&mfree[released % kMeta]);
        }
        if (progressed) {
          idle = 0;
        } else if ((++idle & 0xff) == 0) {
          if (idle > kSpinPolls) {
            set_error(p.err, kErrTimeout);
            *abort_flag = 1;
          }
          if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
        }
      }
      if (landed > 0) {   // products and arrivals in flight end before the CTA does
        commit_by(lead, drain);
        mbar_wait(drain, 0, p.err);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------------------------------------------ softmax
    const int s = warp >> 2, wq = warp & 3;
    const int trow = wq * 32 + lane;   // row of the stream's 128
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lanes + 128 * s;
    const float scale2 = rsqrtf(static_cast<float>(D)) * kLog2e;
    {   // the first segment's queries, while its pages are on their way
      Walker walk(p, pl);
      Segment f;
      if (walk.next(f)) {
        load_queries<D>(p, f, 0, min(f.rows, 128), Qs, tid, 256);
        if (f.rows > 128) load_queries<D>(p, f, 128, f.rows - 128, Qs + L::UNIT, tid, 256);
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&qfull[0]);
          if (f.rows > 128) mbar_arrive(&qfull[1]);
        }
      }
    }
    float m = -INFINITY, l = 0.0f;
    int cnt = 0, had = 0, joins = 0, ends = 0;
    for (int ti = 0;; ++ti) {
      const int mi = ti % kMeta;
      if (!wait(&mfull[mi], ti / kMeta)) break;
      const TileInfo f = info[mi];
      __syncwarp();
      if (lane == 0) mbar_arrive(&mfree[mi]);
      if (!(f.flags & kValid)) break;
      if (f.flags & kFirst) {
        m = -INFINITY;
        l = 0.0f;
        had = 0;
      }
      const bool two = (f.flags & kTwo) != 0;
      const int ntok = f.tp & 0xff, pages = f.tp >> 8;
      const int base = two ? 128 * s : 0;
      const bool active = base + wq * 32 < f.rows;
      if (two || (f.idx & 1) == s) {
        if (!wait(&sfull[s], cnt)) break;
        tc_fence_after();
        if (active) {
          const bool whole = ntok == kTileTok && pages == 0xff;
          auto hide = [&](float *x, int c) {   // columns 32 c .. 32 c + 31: tokens past the end or on no page
            if (whole) return;
            const int n = ntok - 32 * c;
            uint32_t see = n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1 : 0u;
            see &= (((pages >> (2 * c)) & 1) ? 0xffffu : 0u) | (((pages >> (2 * c + 1)) & 1) ? 0xffff0000u : 0u);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = (see >> i) & 1 ? x[i] : -INFINITY;
          };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float x[32];
            tmem_ld32(tS + 32 * c, x);
            tmem_wait_ld();
            hide(x, c);
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx = max3(mx, x[i], x[i + 1]);
          }
          mx *= scale2;
          if (had == 0) {
            m = mx;
          } else if (__any_sync(0xffffffffu, mx > m + kRescale && base + trow < f.rows)) {
            // (rows past the block's are products of whatever an earlier block left in the buffer: they have no say)
            const float mn = fmaxf(m, mx);
            const float a = m == -INFINITY ? 0.0f : exp2f(m - mn);
            l *= a;
            m = mn;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float x[32];
              tmem_ld32(tmem + lanes + 256 + 128 * s + c, x);
              tmem_wait_ld();
              uint32_t y[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(x[i] * a);
              tmem_st16(tmem + lanes + 256 + 128 * s + c, y);
              tmem_st16(tmem + lanes + 256 + 128 * s + c + 16, y + 16);
            }
          }
          const float ms = m == -INFINITY ? 0.0f : m;
          F2 sum = f2(0.0f, 0.0f);
          const F2 sc = f2(scale2, scale2), sub = f2(-ms, -ms);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float x[32];
            tmem_ld32(tS + 32 * c, x);
            tmem_wait_ld();
            hide(x, c);
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float a, b;
              split(fma2(f2(x[2 * i], x[2 * i + 1]), sc, sub), a, b);
              a = fast_exp2(a);
              b = fast_exp2(b);
              sum = add2(sum, f2(a, b));
              const __nv_bfloat162 q = __floats2bfloat162_rn(a, b);
              y[i] = *reinterpret_cast<const uint32_t *>(&q);
            }
            tmem_st16(tS + 16 * c, y);
          }
          float l0, l1;
          split(sum, l0, l1);
          l += l0 + l1;
          tmem_wait_st();
        }
        if (ntok % kPage) {   // rows of the last page past the end: their weights are zero, their values may be anything
          const int vu = 2 * ti + 1;
          if (!wait(&full[vu % NU], vu / NU)) break;
          unsigned char *v = ring + (vu % NU) * L::UNIT;
          const int rows = kPage - ntok % kPage;
          for (int c = wq * 32 + lane; c < rows * (D / 8); c += 128) {
            const int row = ntok + c / (D / 8), k = c % (D / 8);
            *reinterpret_cast<uint4 *>(v + (row >> 3) * L::GROUP + (k >> 3) * 1024 + (row & 7) * 128 + (k & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[s]);
        ++cnt;
        had = 1;
      }
      if (!(f.flags & kLast)) continue;
      const int kind = (f.flags & kKind) ? 1 : 0;
      const bool later = (f.flags & kLater) != 0;
      if (had && !wait(&ofull[s], ends++)) break;
      tc_fence_after();
      Entry x;
      x.q0 = f.q0;
      if (two) {
        const int row = base + trow;
        const bool mine = row < f.rows;
        const Place pp = place<D>(p, x, kind, f.h, f.n0 + min(row, f.rows - 1), later, blockIdx.x);
        if (mine) *pp.ml = make_float2(m, l);
        if (active) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(tmem + lanes + 256 + 128 * s + c, o);
            tmem_wait_ld();
            if (mine)
#pragma unroll
              for (int i = 0; i < 32; i += 8) store32(pp.o + c + i, o + i);
          }
        }
        tc_fence_before();
      } else {
        // the two streams' sums of the same rows: each joins half of the columns
        xm[s * 128 + trow] = m;
        if (s == 1) xm[256 + trow] = l;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(xready);
        if (!wait(xready, joins)) break;
        tc_fence_after();
        const float m0 = xm[trow], m1 = xm[128 + trow], l1 = xm[256 + trow];
        const float M = fmaxf(m0, m1);
        // a stream that saw no token adds nothing (one that saw only NaN has no maximum either, but a sum)
        const bool none0 = m0 == -INFINITY, none1 = m1 == -INFINITY;
        const float w0 = none0 ? 0.0f : exp2f(m0 - M), w1 = none1 ? 0.0f : exp2f(m1 - M);
        const bool mine = trow < f.rows;
        const Place pp = place<D>(p, x, kind, f.h, f.n0 + min(trow, f.rows - 1), later, blockIdx.x);
        if (mine && s == 0) *pp.ml = make_float2(M, l * w0 + l1 * w1);
        if (active) {
#pragma unroll 1
          for (int c = s * (D / 2); c < (s + 1) * (D / 2); c += 32) {
            float o0[32], o1[32];
            tmem_ld32(tmem + lanes + 256 + c, o0);
            tmem_ld32(tmem + lanes + 384 + c, o1);
            tmem_wait_ld();
            if (mine)
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                float r[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) r[k] = (none0 ? 0.0f : o0[i + k] * w0) + (none1 ? 0.0f : o1[i + k] * w1);
                store32(pp.o + c + i, r);
              }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(xdone);
        if (!wait(xdone, joins)) break;
        tc_fence_after();
        ++joins;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// --------------------------------------------------------------------------------------------- joining the records
// The last i in [0, n) with a[i] <= key (0 if there is none), by the whole warp: 32 places at a time.
__device__ __forceinline__ int find_last(const int32_t *a, int n, int key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;   // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && a[min(at, hi - 1)] <= key);
    const int k = le ? 31 - __clz(le) : 0;   // rising entries: the lanes up to k
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The N consecutive elements of a lane, as one load.
template <int N> __device__ __forceinline__ void lane_load(const __nv_bfloat16 *p, float *v) {
  uint32_t w[N / 2];
  if (N == 4) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    w[0] = u.x;
    w[N / 2 - 1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int N> __device__ __forceinline__ void lane_load(const float *p, float *v) {
  if (N == 4) {
    const float4 u = *reinterpret_cast<const float4 *>(p);
    v[0] = u.x, v[1] = u.y, v[N - 2] = u.z, v[N - 1] = u.w;
  } else {
    const float2 u = *reinterpret_cast<const float2 *>(p);
    v[0] = u.x, v[1] = u.y;
  }
}

// One warp a query row: the window's tokens up to itself, and its records of the prefix and of the own context. All but
// the records is older than the first kernel, so it is done before that kernel's end is waited for.
template <class T, int D>
__global__ void __launch_bounds__(128) shared_join_kernel(const HParams p) {
  constexpr int PL = D / 32;  // consecutive dims of a lane
  constexpr int CH = 8;       // records, and WT window tokens, whose loads are in flight together
  constexpr int WT = 4;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  // rows outside the windows (a batch padded to total_q) are left as they are
  const bool live = wid < static_cast<int64_t>(p.total_q) * p.hq && wid >= static_cast<int64_t>(p.q_offsets[0]) * p.hq &&
                    wid < static_cast<int64_t>(p.q_offsets[p.R]) * p.hq;
  float m = -INFINITY, l = 0.0f, o[PL];
#pragma unroll
  for (int k = 0; k < PL; ++k) o[k] = 0.0f;
  int t = 0, hq = 0, h = 0, ent[2] = {-1, -1};
  int64_t at[2] = {0, 0}, end[2] = {0, 0};   // from the entry's start: the item's first tile and its last one's start
  int q0[2] = {0, 0}, row[2] = {0, 0};
  if (live) {
    t = static_cast<int>(quotient(wid, p.hq));
    hq = static_cast<int>(wid - static_cast<int64_t>(t) * p.hq);
    h = hq / p.G;
    float qv[PL];
    lane_load<PL>(static_cast<const T *>(p.q) + (static_cast<size_t>(t) * p.hq + hq) * D + lane * PL, qv);
    const float scale = rsqrtf(static_cast<float>(D)) * kLog2e;
#pragma unroll
    for (int k = 0; k < PL; ++k) qv[k] *= scale;
    const int r = find_last(p.q_offsets, p.R, t);
    const int start = p.q_start[r], past = p.max_pages * kPage;
    if (start > past && lane == 0) set_error(p.err, kErrPage);   // context past the table's end
    const int pos0 = max(start, 0), page0 = pos0 / kPage;
    int pos1 = start > past ? -1 : start + (t - p.q_offsets[r]);
    // the window's pages, one a lane: 64 tokens lie on no more than 5
    if (pos1 / kPage - page0 > 31) {
      if (lane == 0) set_error(p.err, kErrLength);
      pos1 = (page0 + 32) * kPage - 1;
    }
    int my_page = -1;
    if (lane <= pos1 / kPage - page0 && page0 + lane < p.max_pages)
      my_page = p.bt[static_cast<size_t>(r) * p.max_pages + page0 + lane];
    for (int base = pos0; base <= pos1; base += WT) {
      float kv[WT][PL], vv[WT][PL], s[WT];
#pragma unroll
      for (int c = 0; c < WT; ++c) {
        const int pos = min(base + c, pos1);
        const int pg = __shfl_sync(0xffffffffu, my_page, pos / kPage - page0);
        const bool ok = pg >= 0 && pg < p.num_pages;
        s[c] = ok && base + c <= pos1 ? 0.0f : -INFINITY;
        if (!ok && lane == 0) set_error(p.err, kErrPage);
        const size_t off = ((static_cast<size_t>(ok ? pg : 0) * p.hkv + h) * kPage + pos % kPage) * D + lane * PL;
        lane_load<PL>(static_cast<const T *>(p.K) + off, kv[c]);
        lane_load<PL>(static_cast<const T *>(p.V) + off, vv[c]);
      }
      float mn = m;
#pragma unroll
      for (int c = 0; c < WT; ++c) {
        float x = 0.0f;
#pragma unroll
        for (int k = 0; k < PL; ++k) x = fmaf(qv[k], kv[c][k], x);
        x = warp_sum(x);
        if (s[c] == 0.0f) s[c] = x;
        mn = fmaxf(mn, s[c]);
      }
      const float a = m == -INFINITY ? 0.0f : exp2f(m - mn);
      l *= a;
#pragma unroll
      for (int k = 0; k < PL; ++k) o[k] *= a;
#pragma unroll
      for (int c = 0; c < WT; ++c) {
        if (s[c] == -INFINITY) continue;   // no token, or of weight zero
        const float w = exp2f(s[c] - mn);
        l += w;
#pragma unroll
        for (int k = 0; k < PL; ++k) o[k] = fmaf(w, vv[c][k], o[k]);
      }
      m = mn;
    }
    const Groups gr{p.group_off};
    const int g = p.num_groups > 0 ? find_last(p.group_off, p.num_groups, r) : -1;
    const bool in = g >= 0 && gr.off[g] <= r && r < gr.off[g + 1];
    const int shared = in ? shared_pages(p, gr.off, g) : 0;
    if (shared > 0 && shared * kPage <= start) ent[0] = g;
    ent[1] = p.num_groups + r;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
      if (ent[kind] >= 0) {
        const Entry x = entry(p, gr, ent[kind]);
        if (x.tiles == 0) {
          ent[kind] = -1;
          continue;
        }
        q0[kind] = x.q0;
        row[kind] = (t - x.q0) * p.G + hq - h * p.G;
        if (row[kind] < 0 || row[kind] >= x.rows) {   // offsets out of order: the row is none of the group's
          if (lane == 0) set_error(p.err, kErrLength);
          ent[kind] = -1;
          continue;
        }
        const int block = row[kind] / p.block;
        at[kind] = x.first_tile(p, h, block);
        end[kind] = at[kind] + static_cast<int64_t>(x.tiles - 1) * x.cost(p, block);
      }
  }
  grid_dependency_sync();
  if (!live) return;
  const int64_t total = p.start[p.num_groups + p.R];
  const int nb = parts(p, total);
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    if (ent[kind] < 0) continue;
    const int64_t es = p.start[ent[kind]];
    const int b0 = owner_cta(es + at[kind], total, nb), b1 = owner_cta(es + end[kind], total, nb);
    Entry x;
    x.q0 = q0[kind];
    auto take = [&](auto size, int c0) {   // a chunk's records: all loads first, then one step for all
      constexpr int CH = decltype(size)::value;
      float2 ml[CH];
      float rec[CH][PL];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int b = min(c0 + c, b1);
        const Place pp = place<D>(p, x, kind, h, row[kind], b > b0, b);
        ml[c] = __ldcg(pp.ml);
        if (PL == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4 *>(pp.o + lane * PL));
          rec[c][0] = v.x, rec[c][1] = v.y, rec[c][PL - 2] = v.z, rec[c][PL - 1] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2 *>(pp.o + lane * PL));
          rec[c][0] = v.x, rec[c][1] = v.y;
        }
      }
      float mn = m;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (c0 + c <= b1) mn = fmaxf(mn, ml[c].x);
      const float a = m == -INFINITY ? 0.0f : exp2f(m - mn);
      l *= a;
#pragma unroll
      for (int k = 0; k < PL; ++k) o[k] *= a;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        // a record that saw nothing is (-infinity, 0); one that saw only NaN has a sum
        if (c0 + c > b1 || (ml[c].x == -INFINITY && ml[c].y == 0.0f)) continue;
        const float w = exp2f(ml[c].x - mn);
        l = fmaf(ml[c].y, w, l);
#pragma unroll
        for (int k = 0; k < PL; ++k) o[k] = fmaf(rec[c][k], w, o[k]);
      }
      m = mn;
    };
    int c0 = b0;
    for (; c0 + 2 <= b1; c0 += CH) take(std::integral_constant<int, CH>(), c0);
    if (c0 <= b1) take(std::integral_constant<int, 2>(), c0);   // one or two are left: most own contexts
  }
  T *op = static_cast<T *>(p.out) + (static_cast<size_t>(t) * p.hq + hq) * D + lane * PL;
  const bool none = l == 0.0f && m == -INFINITY;
#pragma unroll
  for (int k = 0; k < PL; ++k) op[k] = from_f<T>(none ? 0.0f : o[k] / l);
  if (lane == 0) p.lse[static_cast<size_t>(t) * p.hq + hq] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Parts of the workspace start on multiples of 256 bytes, whatever its address: records are stored 32 bytes at a time.
constexpr size_t kPart = 256;
size_t up(size_t b) { return (b + kPart - 1) / kPart * kPart; }

template <class T, int D> cudaError_t launch_join(const HParams &p, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(p.total_q) * p.hq;
  return launch_pdl(shared_join_kernel<T, D>, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, s, p);
}

template <class T, int D> cudaError_t launch_plain(HParams p, cudaStream_t s) {
  p.block = kPlainRows;
  const cudaError_t e = launch_pdl(shared_plain_kernel<T, D>, dim3(p.nb), dim3(kPlainThreads), 0, s, p);
  return e == cudaSuccess ? launch_join<T, D>(p, s) : e;
}

template <int D> cudaError_t launch_tc(const PoolArgs &pa, HParams p, cudaStream_t s) {
  p.block = kTcBlock;
  CUtensorMap tmK, tmV;
  if (!make_page_map(&tmK, pa.k, pa.num_pages, pa.hkv, D) || !make_page_map(&tmV, pa.v, pa.num_pages, pa.hkv, D))
    return cudaErrorInvalidValue;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!attr_set[dev & 63]) {
    const cudaError_t e =
        cudaFuncSetAttribute(shared_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::ALLOC);
    if (e != cudaSuccess) return e;
    attr_set[dev & 63] = true;
  }
  const cudaError_t e = launch_pdl(shared_tc_kernel<D>, dim3(p.nb), dim3(kTcThreads), Tc<D>::ALLOC, s, tmK, tmV, p);
  return e == cudaSuccess ? launch_join<__nv_bfloat16, D>(p, s) : e;
}

}  // namespace

size_t shared_workspace_bytes(int R, int hkv, int hq, int d, int total_q, int num_groups) {
  (void)hkv;
  const size_t rows = static_cast<size_t>(total_q) * hq, extra = static_cast<size_t>(kMaxCtas) * kMaxBlock;
  // kPart more: the first part may start that far behind an address that is no multiple of it
  return kPart + up((static_cast<size_t>(num_groups) + R + 1) * 8) + 2 * up(rows * 8) + 2 * up(rows * d * 4) +
         up(extra * 8) + up(extra * d * 4);
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
  unsigned char *w = reinterpret_cast<unsigned char *>(up(reinterpret_cast<uintptr_t>(ws)));
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
  if (pa.dtype == 0) return pa.d == 128 ? launch_tc<128>(pa, p, s) : launch_tc<64>(pa, p, s);
  return pa.d == 128 ? launch_plain<float, 128>(p, s) : launch_plain<float, 64>(p, s);
}

}  // namespace kap
