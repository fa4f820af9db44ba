// k_attn_packed.cu - attention over a pool with packed 4-bit pages (sm_103a): proposal (one query a request, the pages
// of a compact view) and verification (a causal window, the whole block table; windows of one row are plain decode).
//
// Mathematics. With code c, scale s and lowest value l of a group of 64 dims, a logit is
//   sum_blocks ( s_k * sum_i q_i c_i + l_k * sum_i q_i ),
// so the inner product runs over the bare codes and the parameters join it once per token and block, in fp32; and
//   out = sum_tokens p v = sum_tokens (p s_v) c + sum_tokens p l_v,
// so p s_v (rounded to fp16, 2^-11) meets the bare codes and the second sum is one number per block and query.
// A code in the low bits of an fp16 is the subnormal c * 2^-24, or c * 2^-20 four bits further up: masking a word of
// codes gives tensor-core operands with no conversion and no subtraction. The factor 16 of every second code goes
// into the query (keys) or into the result (values); the power of two comes off the accumulators.
//
// Tile. A page is 16 tokens: the M of mma.m16n8k16. Logits are S^T[16 tokens x 8 queries] = codes . q^T, and
// O^T[16 dims x 8 queries] = codes^T . p^T; p moves from one to the other inside registers (movmatrix). Queries of one
// KV head (G heads x window rows) are the columns, in tiles of 8. Why mma.sync and registers: a (page, head) is 2304
// bytes, 98 SM cycles of HBM at the measured copy rate, and 4096 codes; as 16-bit operands in shared memory for tcgen05
// those would be 8 KiB written and read again. Fragments masked out of the packed words cost 0.6 instructions a pair and
// touch shared memory once. (A tcgen05 form with the key codes in TMEM took 117 us where this took 63, four windows of 4
// over 32768 tokens: its code conversion and its softmax followed one another in the eight warps that its registers allow.)
//
// Split. Rows of up to 16 pages a warp get a CTA each. Otherwise the pages of all (request, KV head) rows form one line
// that is cut into equal shares, one a CTA, and the last CTA to finish a row merges the parts in their order. In either
// case the warps of a CTA take pages in turn, two at a time for independent work, each with its own ring of bulk copies (a
// whole page-head each), its own references and accumulators; they are joined at the end of a row's part, while the next
// part's queries, ids and first pages are on their way.
//
// Statistics. A warp keeps a reference per query column (at most 2^8 below the running maximum) and one for the value
// scales (at most 2^6 below the largest), so that p s_v stays inside fp16; both move only when a page exceeds them. Values
// of 16-bit pages count for the second one only where sums over it could leave fp32. A token that part of a window does not
// see has probability 0 there; values of such a token that are not finite go round the products.
//
// Bound by the latency of a warp's dependent steps (logits, maximum, exponents, transpose, products), not by HBM and not by
// issue: with 16 warps an SM (one column tile) or 8 the waits of one are not filled by the others. On a GB300, 8 KV heads of
// 128 dims, cycles at 2070 MHz of the whole launch a page and SM, of which HBM would take 107 at the measured copy rate:
//   8 requests of 40960 tokens, 4 columns: 87 us, 4.35 TB/s, 64%: 167 cycles, 79 of them issue (316 instructions);
//   4 of 32768, 16 columns: 65 us, 2.34 TB/s, 34%: 311 cycles, 98 (393);
//   1 of 131072, 40 columns: 158 us, 0.96 TB/s, 14%: 759 cycles, 248 (992: two groups of warps);
//   proposals of 8 and of 128 pages: 5.9 and 16.2 us, a chain of dependent loads.
// The kernels of 16 bits a value are faster at the last two shapes (110 us, 12.7 us): packing pays for decode and for
// windows of up to 16 columns. Heads of 128 dims spill: one column tile 64 bytes a thread, three 56, four 460 to 560.
#include "kap_launch.h"
#include "kap_packed.cuh"

#include <algorithm>
#include <type_traits>

namespace kap {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.402823466e38f;  // reference of a column that has seen nothing: no logit in fp32 is below it
constexpr float kMaxSlack = 8.0f;     // log2 units a logit may exceed its reference by
constexpr float kScaleSlack = 64.0f;  // factor a value scale may exceed its reference by

constexpr int kMaxCtas = 320;  // records of a launch beside one per row: CTAs of the widest grid
// The workspace begins with a counter a CTA, whatever the call's sizes, so that calls of any sizes may take one workspace
// in turn: no call's records lie where another one's counters do.
constexpr size_t kCounterBytes = kMaxCtas * sizeof(int);
static_assert(kCounterBytes % 256 == 0, "records are aligned");

struct AParams {
  const __nv_bfloat16 *k, *v;
  const unsigned char *packed;
  int P16, P4, hkv, hq, R;
  const int32_t *bt;
  int max_pages;
  const int32_t *ctx_len, *seq_len;    // proposal
  ViewArgs view;                       // proposal
  const int32_t *q_offsets, *q_start;  // verification
  int max_q, total_q;
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  float *lse;
  int *counters;  // of the shared row that begins in a CTA's share (at most one: the next begins in a later share)
  float2 *ml;     // [slot][columns]
  float *part;    // [slot][columns][d]
  int ncol;       // columns of a record: G * max_q
  int by_row;     // a CTA a row, no shares
  int *err;
};

template <int D, int NTL, int CS>
struct Cfg {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kCtas = NTL == 1 ? 2 : 1;         // resident CTAs an SM
  static constexpr int PW = kWarps / CS;                 // warps that take pages in turn
  static constexpr int N = NTL * CS * 8;                 // query columns
  static constexpr int NB = D / 64;
  static constexpr int KS = NB * 4;                      // k-steps of the logits
  static constexpr int kQPer = (N * (D / 8) + kThreads - 1) / kThreads;  // 8-dim pieces of the queries a thread takes
  static constexpr int kChunk = PackedChunk<D>::BYTES;
  static constexpr int kStages = (D == 64 ? 8 : NTL == 1 ? 4 : 5) * CS;
  static constexpr bool kPairs = NTL <= 2;               // two pages at once: more independent work a warp
  static constexpr int kQStride = D + 8;                 // bf16 elements of a raw query row
  static constexpr bool kApart = NTL <= 2;               // joins have memory of their own, beside the ring
  static constexpr int kRing = PW * kStages * kChunk;
  static constexpr int kSlots = (PW + 1) / 2;            // joined warps: the others are added to one of these first
  static constexpr int kColStride = D + 8;               // floats of a joined column
  static constexpr int kJoin = kSlots * N * (kColStride + 2) * 4;
  static constexpr int kMaxGrid = 160 * kCtas;           // CTAs, so parts of a row
  static constexpr int kWeights = kMaxGrid * N * 8;      // (maximum, sum) of every part and column
  static constexpr int kJoinArea = kJoin > kWeights ? kJoin : kWeights;
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_JOIN = kApart ? kRing : 0;
  static constexpr int kArea = kApart ? kRing + kJoinArea : (kRing > kJoinArea ? kRing : kJoinArea);
  static constexpr int OFF_QRAW = (kArea + 127) / 128 * 128;
  static constexpr int OFF_QF = OFF_QRAW + (N * kQStride * 2 + 15) / 16 * 16;  // fp16 fragments [tile][k-step / 2][lane][2]
  static constexpr int OFF_QS = OFF_QF + NTL * CS * KS * 32 * 8;               // [N] scale, [N][NB] block sums
  static constexpr int OFF_BAR = OFF_QS + N * (1 + NB) * 4;
  static constexpr int BYTES = OFF_BAR + PW * kStages * 8;
  static_assert(BYTES <= 227 * 1024 / kCtas, "shared memory");
};

// One row's part: pages [p0, p1) of (request r, head h), whose pages lie at [rb, re) of the line.
struct Seg {
  int r, h, row, p0, p1, nq, qoff, last0, ctx, nsel;
  const int32_t *ids, *lps;
  int64_t rb, re;
};

__device__ __forceinline__ int atom_add_acq_rel_gpu(int *p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
      "%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_bf16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}
// Leaves a page to the producer: the warps of all column groups have read it. Returns whether any of them gave up.
template <int CS, int PW>
__device__ __forceinline__ bool release_page(int pw, bool dead) {
  if (CS == 1) {
    __syncwarp();
    return dead;
  }
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(1 + pw), "r"(32 * CS), "r"(dead ? 1 : 0)
      : "memory");
  return any != 0;
}
// Over the eight lanes that hold one column: lanes l, l ^ 4, l ^ 8, l ^ 16.
__device__ __forceinline__ float column_max(float v) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float column_sum(float v) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Whether a word of parameters, or either of a word's two bf16 values, is an infinity or a NaN.
__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Units are what has a page list of its own: a request (every head walks the same list), or a row of a per-head view.
template <bool kView>
struct Units {
  const AParams &p;
  __device__ __forceinline__ int count() const { return kView ? p.R * p.view.rows_per_seq : p.R; }
  __device__ __forceinline__ int heads() const { return kView && p.view.rows_per_seq > 1 ? 1 : p.hkv; }
  // Window of request r, kept inside the query array whatever the device data say.
  __device__ __forceinline__ int window(int r, int &qoff, bool &bad) const {
    if (kView) {
      qoff = r;
      return 1;
    }
    const int a = p.q_offsets[r], b = p.q_offsets[r + 1];
    qoff = min(max(a, 0), p.total_q);
    const int nq = max(min(b, p.total_q) - qoff, 0);
    bad = a != qoff || b < a || b > p.total_q || nq > p.max_q;
    return min(nq, p.max_q);
  }
  __device__ __forceinline__ int pages(int u, int &bad) const {
    if (kView) {
      const int n = p.view.n_entries[u];
      if (n > p.view.cap) bad |= kErrCapacity;
      return min(max(n, 0), p.view.cap);
    }
    int qoff;
    bool wbad = false;
    const int nq = window(u, qoff, wbad);
    if (wbad) bad |= kErrLength;
    if (nq <= 0) return 0;
    const int64_t end = static_cast<int64_t>(p.q_start[u]) + nq;
    const int64_t n = end <= 0 ? 0 : (end + kPage - 1) / kPage;
    if (n > p.max_pages) bad |= kErrPage;
    return static_cast<int>(min(n, static_cast<int64_t>(p.max_pages)));
  }
};

template <int D, int NTL, int CS, bool kView>
__global__ void __launch_bounds__(Cfg<D, NTL, CS>::kThreads, Cfg<D, NTL, CS>::kCtas) attn_kernel(const AParams p) {
  using C = Cfg<D, NTL, CS>;
  using L = PackedChunk<D>;
  constexpr int NB = C::NB;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_scan[C::kWarps], s_total, s_base;
  __shared__ int s_unit, s_flag;
  __shared__ Seg s_seg;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pw = warp % C::PW, cg = warp / C::PW;  // which pages, which group of NTL column tiles
  const int g = lane >> 2, t = lane & 3;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + pw * C::kStages;
  unsigned char *ring = smem + C::OFF_RING + pw * C::kStages * C::kChunk;
  __nv_bfloat16 *qraw = reinterpret_cast<__nv_bfloat16 *>(smem + C::OFF_QRAW);
  uint4 *qfrag4 = reinterpret_cast<uint4 *>(smem + C::OFF_QF);  // two k-steps
  float *qscale = reinterpret_cast<float *>(smem + C::OFF_QS);
  float *qsum = qscale + C::N;

  if (cg == 0 && lane < C::kStages) mbar_init(&bars[lane], 1);
  fence_barrier_init();
  grid_dependency_sync();

  // ---- this CTA's share of the line of pages, and the unit that it starts in
  const Units<kView> units{p};
  const int U = units.count(), H = units.heads();
  // Zeros for the heads [h0, h0 + heads) of a request whose rows have no pages.
  auto empty_rows = [&](int r, int h0, int heads) {
    int qoff;
    bool wb = false;
    const int nq = units.window(r, qoff, wb), per = heads * (p.hq / p.hkv);
    for (int i = 0; i < nq * per; ++i) {
      const size_t o = static_cast<size_t>(qoff + i / per) * p.hq + h0 * (p.hq / p.hkv) + i % per;
      p.lse[o] = -INFINITY;
      for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4 *>(p.out + o * D + c) = make_uint4(0, 0, 0, 0);
    }
    if (kView) set_error(p.err, kErrLength);
  };
  // The rest of a part's description; by one thread, into s_seg.
  auto describe = [&](int unit, int head, int p0, int p1, int n, int64_t rb) {
    Seg s;
    s.r = kView ? unit / p.view.rows_per_seq : unit;
    s.h = H == 1 && kView ? unit - s.r * p.view.rows_per_seq : head;
    s.row = s.r * p.hkv + s.h;
    s.p0 = p0;
    s.p1 = p1;
    s.rb = rb;
    s.re = rb + n;
    bool wb = false;
    s.nq = units.window(s.r, s.qoff, wb);
    if (kView) {
      s.last0 = p.seq_len[s.r] - 1;
      s.ctx = p.ctx_len[s.r];
      s.nsel = p.view.n_selected[unit];
      s.ids = p.view.bt + static_cast<size_t>(unit) * p.view.cap;
      s.lps = p.view.lp + static_cast<size_t>(unit) * p.view.cap;
    } else {
      s.last0 = p.q_start[s.r];
      s.ctx = 0;
      s.nsel = 0;
      s.ids = p.bt + static_cast<size_t>(s.r) * p.max_pages;
      s.lps = nullptr;
    }
    s_seg = s;
  };
  int64_t x = 0, x1 = 0, share = 1;
  // The part at x, from the unit at or before it (its pages start at base).
  auto find_part = [&](int unit, int64_t base, int64_t x) {
    int dummy = 0;
    int n = units.pages(unit, dummy);
    while (x >= base + static_cast<int64_t>(n) * H) {
      base += static_cast<int64_t>(n) * H;
      n = units.pages(++unit, dummy);
    }
    const int64_t in = x - base;
    const int head = in < n ? 0 : static_cast<int>(in / n), p0 = static_cast<int>(in - static_cast<int64_t>(head) * n);
    describe(unit, head, p0, static_cast<int>(min(static_cast<int64_t>(n), p0 + (x1 - x))), n, x - p0);
    s_unit = unit;
    s_base = base;
  };
  if (p.by_row) {
    const int unit = blockIdx.x / H, head = blockIdx.x - unit * H;
    int bad = 0;
    const int n = units.pages(unit, bad);
    if (tid == 0) {
      if (bad) set_error(p.err, bad);
      const int r = kView ? unit / p.view.rows_per_seq : unit;
      if (n == 0) empty_rows(r, H == 1 && kView ? unit - r * p.view.rows_per_seq : head, 1);
      else describe(unit, head, 0, n, n, 0);
    }
    if (n == 0) return;
    x1 = share = n;
  } else {
    int64_t total = 0, incl = 0, n_own = 0;
    int bad = 0;
    for (int base = 0; base < U; base += C::kThreads) {
      const int u = base + tid;
      n_own = u < U ? static_cast<int64_t>(units.pages(u, bad)) * H : 0;
      incl = block_inclusive_scan<int64_t>(n_own, s_scan);
      if (tid == C::kThreads - 1) s_total = incl;
      __syncthreads();
      total += s_total;
      __syncthreads();
      if (u < U && n_own == 0 && u % gridDim.x == blockIdx.x) {
        const int r = kView ? u / p.view.rows_per_seq : u;
        empty_rows(r, H == 1 && kView ? u - r * p.view.rows_per_seq : 0, H == 1 && kView ? 1 : p.hkv);
      }
    }
    if (bad && blockIdx.x == 0) set_error(p.err, bad);
    // equal shares, of two pages a warp at least
    share = total < (1 << 30) ? (static_cast<uint32_t>(total) + gridDim.x - 1) / gridDim.x
                              : (total + gridDim.x - 1) / gridDim.x;
    share = max(share, static_cast<int64_t>(2 * C::PW));
    x = share * blockIdx.x;
    x1 = min(x + share, total);
    if (x >= x1) return;
    if (U <= C::kThreads) {  // the scan above still stands
      if (incl - n_own <= x && x < incl) find_part(tid, incl - n_own, x);
    } else {
      int64_t before = 0;
      int dummy = 0;
      for (int base = 0; base < U; base += C::kThreads) {
        const int u = base + tid;
        const int64_t n = u < U ? static_cast<int64_t>(units.pages(u, dummy)) * H : 0;
        const int64_t upto = before + block_inclusive_scan<int64_t>(n, s_scan);
        if (upto - n <= x && x < upto) find_part(u, upto - n, x);
        if (tid == C::kThreads - 1) s_total = upto;
        __syncthreads();
        before = s_total;
        __syncthreads();
        if (before > x) break;
      }
    }
  }
  __syncthreads();
  Seg s = s_seg;

  const int G = p.hq / p.hkv;
  const float qk = rsqrtf(static_cast<float>(D)) * kLog2e;
  const int tokA = (g >> 1) + 4 * (g & 1), tokB = tokA + 8;  // tokens of this lane's two logit rows
  uint32_t issued = 0, consumed = 0;               // packed pages copied and used by this warp
  uint32_t in_st = 0, out_st = 0, out_parity = 0;  // their ring slots
  bool dead = false;
  auto advance = [&]() {
    ++consumed;
    if (++out_st == C::kStages) {
      out_st = 0;
      out_parity ^= 1;
    }
  };

  // This warp's items of a part: pages p0 + pw, p0 + pw + PW, ...; ids of 32 items a load, two loads held.
  int nit = 0, idc = -1, lpc = 0, idn = -1, lpn = 0, batch = 0, ahead = 0;
  unsigned m4c = 0u, m4n = 0u, whole = 0u;  // packed pages of the two loads; those of the first that every column sees in full
  auto load_ids = [&](int b, int &id, int &lp) {
    const int j = b * 32 + lane;
    id = -1;
    lp = 0;
    if (j < nit) {
      const int e = s.p0 + pw + C::PW * j;
      id = s.ids[e];
      if (kView) lp = s.lps[e];
    }
  };
  auto is_packed = [&](int id) { return id >= p.P16 && id < p.P16 + p.P4; };
  auto classify = [&]() {
    const int e = s.p0 + pw + C::PW * (batch * 32 + lane);
    const int pos0 = (kView ? lpc : e) * kPage, first = kView && e >= s.nsel ? s.ctx : 0;
    m4c = __ballot_sync(0xffffffffu, is_packed(idc));
    m4n = __ballot_sync(0xffffffffu, is_packed(idn));
    whole = m4c & __ballot_sync(0xffffffffu, pos0 + kPage - 1 <= s.last0 && pos0 >= first);
  };
  auto open_part = [&]() {
    nit = s.p1 - s.p0 > pw ? (s.p1 - s.p0 - pw + C::PW - 1) / C::PW : 0;
    batch = 0;
    ahead = 0;
    load_ids(0, idc, lpc);
    load_ids(1, idn, lpn);
  };
  // Copies for the items from `ahead` on that are held, as far as the ring has room: the lane that holds an item's id
  // starts its copy, in the slot of its rank among them.
  auto issue_from = [&](unsigned held, int ids, int first_item) {
    const unsigned m = held & (~0u << (ahead - first_item));
    const int room = C::kStages - static_cast<int>(issued - consumed);
    const int rank = __popc(m & ((1u << lane) - 1u));
    const bool mine = (m >> lane & 1) && rank < room;
    if (mine && cg == 0) {
      const int st = in_st + rank < C::kStages ? in_st + rank : in_st + rank - C::kStages;
      mbar_arrive_expect_tx(&bars[st], C::kChunk);
      bulk_g2s(ring + st * C::kChunk, p.packed + (static_cast<size_t>(ids - p.P16) * p.hkv + s.h) * C::kChunk, C::kChunk,
               &bars[st]);
    }
    const unsigned started = __ballot_sync(0xffffffffu, mine);
    const int n = __popc(started);
    issued += n;
    in_st = in_st + n < C::kStages ? in_st + n : in_st + n - C::kStages;
    ahead = first_item + (started == m ? 32 : 32 - __clz(started));  // with room there is a start unless m is empty
  };
  auto issue = [&]() {
    if (issued - consumed >= C::kStages) return;
    if (ahead < (batch + 1) * 32) issue_from(m4c, idc, batch * 32);
    if (ahead >= (batch + 1) * 32 && ahead < (batch + 2) * 32 && issued - consumed < C::kStages)
      issue_from(m4n, idn, (batch + 1) * 32);
  };
  // The queries' loads, asked for before the pages: behind those they would wait for the whole ring.
  uint4 qv[C::kQPer];
  auto load_queries = [&]() {
#pragma unroll
    for (int k = 0; k < C::kQPer; ++k) {
      const int i = tid + k * C::kThreads, c = i / (D / 8), piece = i % (D / 8);
      const int w = c / G, a = c - w * G;
      qv[k] = make_uint4(0, 0, 0, 0);
      if (c < G * s.nq)
        qv[k] = *reinterpret_cast<const uint4 *>(p.q + (static_cast<size_t>(s.qoff + w) * p.hq + s.h * G + a) * D + piece * 8);
    }
  };
  load_queries();
  open_part();
  classify();
  if (!dead) issue();

  while (true) {
    const int M = G * s.nq;
    // ---- queries: a thread takes 8 dims of a column, whose fp16 operands are one entry of the fragment array
#pragma unroll
    for (int k = 0; k < C::kQPer; ++k) {
      const int i = tid + k * C::kThreads, c = i / (D / 8), piece = i % (D / 8);
      if (c < C::N) {  // whole columns: D / 8 neighbouring lanes
        float v[8];
        Vec16<__nv_bfloat16>::unpack(qv[k], v);
        float mx = 0.0f, sum = 0.0f;
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          mx = fmaxf(mx, fabsf(v[z]));
          sum += v[z];
        }
        const unsigned peers = __activemask();
#pragma unroll
        for (int o = D / 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(peers, mx, o));
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(peers, sum, o);
        // largest magnitude to [2^14, 2^15): every bf16 down to 2^-24 of it is exact in fp16, a sixteenth too
        const int e = static_cast<int>((__float_as_uint(mx) >> 23) & 255);
        const int sh = e == 0 || e == 255 ? 0 : min(141 - e, 126);
        const float sc = __uint_as_float(static_cast<uint32_t>(127 + max(sh, -126)) << 23), s16 = sc * 0.0625f;
        if (piece == 0) qscale[c] = sc;
        if ((piece & 7) == 0) qsum[c * NB + (piece >> 3)] = sum * qk;
        *reinterpret_cast<uint4 *>(qraw + c * C::kQStride + piece * 8) = qv[k];
        // piece = 8 b + 2 t + i: dims 64 b + 16 t + 8 i .. + 7, k-steps 4 b + 2 i and the next, lane (c % 8, t)
        qfrag4[((c >> 3) * (C::KS / 2) + (piece >> 3) * 2 + (piece & 1)) * 32 + (c & 7) * 4 + ((piece >> 1) & 3)] =
            make_uint4(pack_f16(v[0] * sc, v[4] * sc), pack_f16(v[1] * s16, v[5] * s16), pack_f16(v[2] * sc, v[6] * sc),
                       pack_f16(v[3] * s16, v[7] * s16));
      }
    }
    __syncthreads();
    const bool more = x + (s.p1 - s.p0) < x1;
    if (more && tid == C::kThreads - 1) find_part(s_unit, s_base, x + (s.p1 - s.p0));  // its loads run beside the pages

    // per column of this lane (two a tile): logit factor, block sums, reference, sum, sum p * lowest
    F2 cq[NTL], qs[NTL][NB], lsum[NTL], lv[NTL][NB];
    float mref[NTL][2], acc[NTL][NB][4][4];
#pragma unroll
    for (int j = 0; j < NTL; ++j) {
      const int col = (cg * NTL + j) * 8 + 2 * t;
      cq[j] = f2(qk * 0x1p24f / qscale[col], qk * 0x1p24f / qscale[col + 1]);
      mref[j][0] = mref[j][1] = kNoMax;
      lsum[j] = f2(0.0f, 0.0f);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        qs[j][b] = f2(qsum[col * NB + b], qsum[(col + 1) * NB + b]);
        lv[j][b] = f2(0.0f, 0.0f);
      }
    }
#pragma unroll
    for (int j = 0; j < NTL; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[j][b][m][c] = 0.0f;
    float inv_e = 1.0f;       // 1 / reference of the value scales, a power of two
    float sv_limit = -1.0f;   // largest scale that it admits; the first packed page sets both

    // A token that some columns see and others do not takes part in the products of all of them, with probability 0 where it
    // is hidden: its values have to be finite there. Those that are not are taken out of the operands and added here, to the
    // columns that see them. value(token, block, dim of the block) is asked for these tokens only; rare.
    auto add_not_finite = [&](int pos0, auto value) {
#pragma unroll 1
      for (int tok = 0; tok < kPage; ++tok) {
        const int pos = pos0 + tok;
        if (pos <= s.last0 || pos > s.last0 + s.nq - 1) continue;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float v = value(tok, b, g * 8 + 2 * m + i);
              if (fabsf(v) < INFINITY) continue;
#pragma unroll
              for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  if (pos <= s.last0 + ((cg * NTL + j) * 8 + 2 * t + c) / G) acc[j][b][m][2 * i + c] += v;
            }
      }
    };

    // Moves the references up where a page's logits (page[n][j][4]) or value scales exceed them by too much, and turns
    // the logits into probabilities over the references (pairs of columns of this lane's two tokens).
    const int last_all = s.last0 + s.nq - 1;
    // scales() is the lane's largest finite value scale, asked for where svmax is infinite.
    auto probabilities = [&](auto np, float (*sc)[NTL][4], float svmax, auto scales, F2 (*pA)[NTL], F2 (*pB)[NTL]) {
      constexpr int NP = decltype(np)::value;
      auto distances = [&]() {
#pragma unroll
        for (int j = 0; j < NTL; ++j) {
          const F2 m = f2(-mref[j][0], -mref[j][1]);
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            pA[n][j] = add2(f2(sc[n][j][0], sc[n][j][1]), m);
            pB[n][j] = add2(f2(sc[n][j][2], sc[n][j][3]), m);
          }
        }
      };
      distances();
      float over = -INFINITY;
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int j = 0; j < NTL; ++j) {
          float a, b, c, d;
          split(pA[n][j], a, b);
          split(pB[n][j], c, d);
          over = fmaxf(over, fmaxf(fmaxf(a, b), fmaxf(c, d)));
        }
      if (__any_sync(0xffffffffu, over > kMaxSlack || svmax > sv_limit)) {
        float ratio = 1.0f;
        const float mx = column_max(svmax < INFINITY ? svmax : scales());  // the lanes of a column hold all tokens
        if (mx > sv_limit) {
          float least = 0x1p-100f;
          if (sv_limit < 0.0f) {  // the first scale: what 16-bit pages have summed up over 1 has to stay in fp32 over it
            float a = 0.0f;
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int z = 0; z < 4; ++z)
#pragma unroll
                  for (int c = 0; c < 4; ++c) a = fmaxf(a, fabsf(acc[j][b][z][c]));
            const uint32_t e = __reduce_max_sync(0xffffffffu, a < INFINITY ? __float_as_uint(a) & 0x7f800000u : 0u);
            least = fmaxf(least, __uint_as_float(e) * 0x1p-100f);
          }
          const float ie = 1.0f / fmaxf(__uint_as_float(__float_as_uint(mx) & 0x7f800000u), least);
          ratio = ie / inv_e;
          inv_e = ie;
          sv_limit = kScaleSlack / ie;
        }
#pragma unroll
        for (int j = 0; j < NTL; ++j) {
          float f[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = mref[j][c];
#pragma unroll
            for (int n = 0; n < NP; ++n) m = fmaxf(m, fmaxf(sc[n][j][c], sc[n][j][2 + c]));
            m = column_max(m);
            f[c] = fast_exp2(mref[j][c] - m);
            mref[j][c] = m;
          }
          const F2 ff = f2(f[0], f[1]);
          lsum[j] = mul2(lsum[j], ff);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            lv[j][b] = mul2(lv[j][b], ff);
#pragma unroll
            for (int z = 0; z < 4; ++z)
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[j][b][z][c] *= f[c & 1] * ratio;
          }
        }
        distances();
      }
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int j = 0; j < NTL; ++j) {
          float a, b, c, d;
          split(pA[n][j], a, b);
          split(pB[n][j], c, d);
          pA[n][j] = f2(fast_exp2(a), fast_exp2(b));
          pB[n][j] = f2(fast_exp2(c), fast_exp2(d));
          lsum[j] = add2(lsum[j], add2(pA[n][j], pB[n][j]));
        }
    };
    // Hides what lies past a column's last token or before `first`.
    auto hide = [&](float (*sc)[4], int pos0, int first) {
      const int pA = pos0 + tokA, pB = pos0 + tokB;
#pragma unroll
      for (int j = 0; j < NTL; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int last = s.last0 + ((cg * NTL + j) * 8 + 2 * t + c) / G;
          if (pA > last || pA < first) sc[j][c] = -INFINITY;
          if (pB > last || pB < first) sc[j][2 + c] = -INFINITY;
        }
    };

    // NP packed pages at once; `edge` (one page only): part of it is hidden from some column.
    auto packed_pages = [&](auto np, const unsigned char *const *chs, bool edge, int pos0, int first) {
      constexpr int NP = decltype(np)::value;
      float sc[NP][NTL][4];
      uint32_t vpA[NP][NB], vpB[NP][NB];
      {
        float sb[NP][NTL][NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t a[NP][4], bb[NP][4];
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            const uint2 wA = *reinterpret_cast<const uint2 *>(chs[n] + b * L::kBlock + tokA * 32 + t * 8);
            const uint2 wB = *reinterpret_cast<const uint2 *>(chs[n] + b * L::kBlock + tokB * 32 + t * 8);
            a[n][0] = wA.x, a[n][1] = wA.x >> 8, a[n][2] = wA.y, a[n][3] = wA.y >> 8;
            bb[n][0] = wB.x, bb[n][1] = wB.x >> 8, bb[n][2] = wB.y, bb[n][3] = wB.y >> 8;
          }
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            uint4 q[NTL];
#pragma unroll
            for (int j = 0; j < NTL; ++j) q[j] = qfrag4[((cg * NTL + j) * (C::KS / 2) + b * 2 + i / 2) * 32 + lane];
#pragma unroll
            for (int n = 0; n < NP; ++n) {
              const uint32_t a0 = a[n][i] & 0x000f000fu, a1 = bb[n][i] & 0x000f000fu, a2 = a[n][i] & 0x00f000f0u,
                             a3 = bb[n][i] & 0x00f000f0u;
              const uint32_t e0 = a[n][i + 1] & 0x000f000fu, e1 = bb[n][i + 1] & 0x000f000fu,
                             e2 = a[n][i + 1] & 0x00f000f0u, e3 = bb[n][i + 1] & 0x00f000f0u;
#pragma unroll
              for (int j = 0; j < NTL; ++j) {
                if (i == 0) mma_f16_zero(sb[n][j][b], a0, a1, a2, a3, q[j].x, q[j].y);
                else mma_f16(sb[n][j][b], a0, a1, a2, a3, q[j].x, q[j].y);
                mma_f16(sb[n][j][b], e0, e1, e2, e3, q[j].z, q[j].w);
              }
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          F2 sA[NB], sB[NB], lA[NB], lB[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t kA = *reinterpret_cast<const uint32_t *>(chs[n] + L::OFF_KPAR + (b * kPage + tokA) * 4);
            const uint32_t kB = *reinterpret_cast<const uint32_t *>(chs[n] + L::OFF_KPAR + (b * kPage + tokB) * 4);
            vpA[n][b] = *reinterpret_cast<const uint32_t *>(chs[n] + L::OFF_VPAR + (b * kPage + tokA) * 4);
            vpB[n][b] = *reinterpret_cast<const uint32_t *>(chs[n] + L::OFF_VPAR + (b * kPage + tokB) * 4);
            sA[b] = f2(param_scale(kA), param_scale(kA)), lA[b] = f2(param_low(kA), param_low(kA));
            sB[b] = f2(param_scale(kB), param_scale(kB)), lB[b] = f2(param_low(kB), param_low(kB));
          }
#pragma unroll
          for (int j = 0; j < NTL; ++j) {
            F2 a = mul2(f2(sb[n][j][0][0], sb[n][j][0][1]), sA[0]), b = mul2(f2(sb[n][j][0][2], sb[n][j][0][3]), sB[0]);
            F2 la = mul2(lA[0], qs[j][0]), lb = mul2(lB[0], qs[j][0]);
#pragma unroll
            for (int z = 1; z < NB; ++z) {
              a = fma2(f2(sb[n][j][z][0], sb[n][j][z][1]), sA[z], a);
              b = fma2(f2(sb[n][j][z][2], sb[n][j][z][3]), sB[z], b);
              la = fma2(lA[z], qs[j][z], la);
              lb = fma2(lB[z], qs[j][z], lb);
            }
            split(fma2(a, cq[j], la), sc[n][j][0], sc[n][j][1]);
            split(fma2(b, cq[j], lb), sc[n][j][2], sc[n][j][3]);
          }
        }
      }
      bool odd = false;  // tokens that some columns do not see have parameters that are not finite
      if (NP == 1 && edge) {
        hide(sc[0], pos0, first);
        // a token that no column sees: its parameters may hold anything
        const bool hA = pos0 + tokA > last_all || pos0 + tokA < first, hB = pos0 + tokB > last_all || pos0 + tokB < first;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (hA) vpA[0][b] = 0u;
          if (hB) vpB[0][b] = 0u;
        }
        if (!kView) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const bool oA = pos0 + tokA > s.last0 && not_finite(vpA[0][b]), oB = pos0 + tokB > s.last0 && not_finite(vpB[0][b]);
            if (oA) vpA[0][b] = 0u;
            if (oB) vpB[0][b] = 0u;
            odd |= oA || oB;
          }
          odd = __any_sync(0xffffffffu, odd) != 0;
        }
      }
      float svmax = 0.0f;
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int b = 0; b < NB; ++b) svmax = fmaxf(svmax, fmaxf(param_scale(vpA[n][b]), param_scale(vpB[n][b])));
      F2 pA[NP][NTL], pB[NP][NTL];
      auto scales = [&]() {
        float m = 0.0f;
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const float a = param_scale(vpA[n][b]), c = param_scale(vpB[n][b]);
            m = fmaxf(m, fmaxf(a < INFINITY ? a : 0.0f, c < INFINITY ? c : 0.0f));
          }
        return m;
      };
      probabilities(np, sc, svmax, scales, pA, pB);
      if (!kView && odd)
        add_not_finite(pos0, [&](int tok, int b, int x) {
          const uint32_t par = *reinterpret_cast<const uint32_t *>(chs[0] + L::OFF_VPAR + (b * kPage + tok) * 4);
          const int two = chs[0][L::OFF_V + b * L::kBlock + tok * 32 + x / 2];
          return fmaf(param_scale(par), static_cast<float>(x & 1 ? two >> 4 : two & 15), param_low(par));
        });
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          const float fA = param_low(vpA[n][b]), fB = param_low(vpB[n][b]);
          const float ea = param_scale(vpA[n][b]) * inv_e, eb = param_scale(vpB[n][b]) * inv_e;
          const F2 lA = f2(fA, fA), lB = f2(fB, fB), eA = f2(ea, ea), eB = f2(eb, eb);
          uint32_t pb[NTL][2];
#pragma unroll
          for (int j = 0; j < NTL; ++j) {
            lv[j][b] = fma2(pA[n][j], lA, fma2(pB[n][j], lB, lv[j][b]));
            float x, y;
            split(mul2(pA[n][j], eA), x, y);
            pb[j][0] = transpose8x8(pack_f16(x, y));
            split(mul2(pB[n][j], eB), x, y);
            pb[j][1] = transpose8x8(pack_f16(x, y));
          }
          const unsigned char *vb = chs[n] + L::OFF_V + b * L::kBlock + g * 4;
          const uint32_t v0 = *reinterpret_cast<const uint32_t *>(vb + t * 32);
          const uint32_t v1 = *reinterpret_cast<const uint32_t *>(vb + (t + 4) * 32);
          const uint32_t v2 = *reinterpret_cast<const uint32_t *>(vb + (t + 8) * 32);
          const uint32_t v3 = *reinterpret_cast<const uint32_t *>(vb + (t + 12) * 32);
          const uint32_t x0 = __byte_perm(v0, v1, 0x5410), x1w = __byte_perm(v0, v1, 0x7632);
          const uint32_t y0 = __byte_perm(v2, v3, 0x5410), y1w = __byte_perm(v2, v3, 0x7632);
          const uint32_t xs[4] = {x0, x0 >> 8, x1w, x1w >> 8}, ys[4] = {y0, y0 >> 8, y1w, y1w >> 8};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t a0 = xs[m] & 0x000f000fu, a1 = xs[m] & 0x00f000f0u, a2 = ys[m] & 0x000f000fu,
                           a3 = ys[m] & 0x00f000f0u;
#pragma unroll
            for (int j = 0; j < NTL; ++j) mma_f16(acc[j][b][m], a0, a1, a2, a3, pb[j][0], pb[j][1]);
          }
        }
      }
    };

    // One 16-bit page, straight from global memory: these are the few a view's or a table's tail has.
    auto page16 = [&](int id, bool edge, int pos0, int first) {
      float sc[1][NTL][4];
      const __nv_bfloat16 *kp = p.k + (static_cast<size_t>(id) * p.hkv + s.h) * (kPage * D);
#pragma unroll
      for (int j = 0; j < NTL; ++j) sc[0][j][0] = sc[0][j][1] = sc[0][j][2] = sc[0][j][3] = 0.0f;
#pragma unroll
      for (int z = 0; z < D / 32; ++z) {
        const uint4 kA = *reinterpret_cast<const uint4 *>(kp + tokA * D + z * 32 + t * 8);
        const uint4 kB = *reinterpret_cast<const uint4 *>(kp + tokB * D + z * 32 + t * 8);
#pragma unroll
        for (int j = 0; j < NTL; ++j) {
          const uint4 q = *reinterpret_cast<const uint4 *>(qraw + ((cg * NTL + j) * 8 + g) * C::kQStride + z * 32 + t * 8);
          mma_bf16(sc[0][j], kA.x, kB.x, kA.y, kB.y, q.x, q.y);
          mma_bf16(sc[0][j], kA.z, kB.z, kA.w, kB.w, q.z, q.w);
        }
      }
#pragma unroll
      for (int j = 0; j < NTL; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[0][j][c] *= qk;
      if (edge) hide(sc[0], pos0, first);
      const __nv_bfloat16 *vp = p.v + (static_cast<size_t>(id) * p.hkv + s.h) * (kPage * D);
      // Sums of values over a very small reference (of packed pages that hold next to nothing) might leave fp32: 2^-40 of
      // the page's largest value then counts as a value scale. A packed token loses 2^-65 of that value at most.
      float svmax = -INFINITY;
      if (sv_limit >= 0.0f && inv_e > 0x1p20f) {
        uint32_t m = 0u;
#pragma unroll 1
        for (int i = lane; i < kPage * D; i += 32) {
          const uint32_t a = reinterpret_cast<const unsigned short *>(vp)[i] & 0x7fffu;
          if (a < 0x7f80u && pos0 + i / D <= last_all && pos0 + i / D >= first) m = max(m, a);
        }
        svmax = __uint_as_float(__reduce_max_sync(0xffffffffu, m) << 16) * 0x1p-40f;
      }
      F2 pA[1][NTL], pB[1][NTL];
      probabilities(std::integral_constant<int, 1>{}, sc, svmax, []() { return 0.0f; }, pA, pB);
      // p as two bf16 terms, in the accumulators' unit (2^-24 of the value over the scale reference): a reference below 1
      // goes into p, one above 1 into the values, so that neither leaves the normal numbers
      const float unit16 = 0x1p-24f * fmaxf(inv_e, 1.0f), vunit = fminf(inv_e, 1.0f);
      uint32_t ph[NTL][2], pl[NTL][2];
#pragma unroll
      for (int j = 0; j < NTL; ++j)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float u0, u1;
          split(z ? pB[0][j] : pA[0][j], u0, u1);
          u0 *= unit16, u1 *= unit16;
          const uint32_t hi = pack_bf16(u0, u1);
          pl[j][z] = transpose8x8(pack_bf16(u0 - __uint_as_float(hi << 16), u1 - __uint_as_float(hi & 0xffff0000u)));
          ph[j][z] = transpose8x8(hi);
        }
      bool see[4], part[4], odd = false;  // rows that no column sees, or not every one, may hold anything
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int pos = pos0 + t + 4 * z;
        see[z] = pos <= last_all && pos >= first;
        part[z] = !kView && pos > s.last0;
      }
      const __nv_bfloat162 even = __floats2bfloat162_rn(vunit, vunit),
                           high = __floats2bfloat162_rn(16.0f * vunit, 16.0f * vunit);
      auto times = [](uint32_t w, __nv_bfloat162 f) {  // by a power of two: exact
        const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w), f);
        return *reinterpret_cast<const uint32_t *>(&r);
      };
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint4 w[4];
#pragma unroll
        for (int z = 0; z < 4; ++z)
          w[z] = see[z] ? *reinterpret_cast<const uint4 *>(vp + (t + 4 * z) * D + b * 64 + g * 8) : make_uint4(0, 0, 0, 0);
        if (!kView && edge) {
#pragma unroll
          for (int z = 0; z < 4; ++z)
            if (part[z] && (not_finite(w[z].x) || not_finite(w[z].y) || not_finite(w[z].z) || not_finite(w[z].w))) {
              odd = true;
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                uint32_t &u = (&w[z].x)[m];
                if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
                if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
              }
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t u[4] = {(&w[0].x)[m], (&w[1].x)[m], (&w[2].x)[m], (&w[3].x)[m]};
          const uint32_t a0 = times(__byte_perm(u[0], u[1], 0x5410), even), a2 = times(__byte_perm(u[2], u[3], 0x5410), even);
          const uint32_t a1 = times(__byte_perm(u[0], u[1], 0x7632), high), a3 = times(__byte_perm(u[2], u[3], 0x7632), high);
#pragma unroll
          for (int j = 0; j < NTL; ++j) {
            mma_bf16(acc[j][b][m], a0, a1, a2, a3, ph[j][0], ph[j][1]);
            mma_bf16(acc[j][b][m], a0, a1, a2, a3, pl[j][0], pl[j][1]);
          }
        }
      }
      if (!kView && edge && __any_sync(0xffffffffu, odd))
        add_not_finite(pos0, [&](int tok, int b, int x) { return __bfloat162float(vp[tok * D + b * 64 + x]); });
    };

    // Waits for the next page of the ring; false (for every lane) when the wait ran out.
    auto arrived = [&]() { return __all_sync(0xffffffffu, mbar_wait(&bars[out_st], out_parity, p.err)) != 0; };
    for (int k = 0; k < nit;) {
      if ((k >> 5) != batch) {
        idc = idn;
        lpc = lpn;
        load_ids(++batch + 1, idn, lpn);
        classify();
      }
      if (!dead) issue();
      const int kk = k & 31;
      if (whole >> kk & 1) {
        const bool two = C::kPairs && (whole >> kk & 3) == 3;
        if (!dead) {
          const unsigned char *chs[2] = {ring + out_st * C::kChunk, nullptr};
          bool ok = arrived();
          if (ok) advance();
          if (ok && two) {
            chs[1] = ring + out_st * C::kChunk;
            ok = arrived();
            if (ok) {
              advance();
              packed_pages(std::integral_constant<int, 2>{}, chs, false, 0, 0);
            }
          } else if (ok) {
            packed_pages(std::integral_constant<int, 1>{}, chs, false, 0, 0);
          }
          dead = release_page<CS, C::PW>(pw, !ok);  // from then on nothing is read; what is in flight is waited for below
        }
        k += two ? 2 : 1;
        continue;
      }
      const int id = __shfl_sync(0xffffffffu, idc, kk);
      const int e = s.p0 + pw + C::PW * k;
      const int pos0 = (kView ? __shfl_sync(0xffffffffu, lpc, kk) : e) * kPage, first = kView && e >= s.nsel ? s.ctx : 0;
      ++k;
      if (m4c >> kk & 1) {
        if (dead) continue;
        const unsigned char *chs[1] = {ring + out_st * C::kChunk};
        const bool ok = arrived();
        if (ok) {
          advance();
          packed_pages(std::integral_constant<int, 1>{}, chs, true, pos0, first);
        }
        dead = release_page<CS, C::PW>(pw, !ok);
      } else if (id >= 0 && id < p.P16) {
        page16(id, pos0 + kPage - 1 > s.last0 || pos0 < first, pos0, first);
      } else if (lane == 0) {
        set_error(p.err, kErrPage);
      }
    }
    // a wait that ran out leaves copies in flight: each is waited for (with a limit) before its slot's memory is reused
    if (dead) {
      while (consumed != issued) {
        mbar_wait(&bars[out_st], out_parity, p.err);
        advance();
      }
    }

    // ---- values in their own unit, columns summed over their lanes
    // 2^24 and the scale reference: in two factors, as their product may leave fp32 (and an accumulator times 2^24 where the
    // reference is small)
    const float unit_e = 0x1p24f / fmaxf(inv_e, 1.0f), unit_v = 1.0f / fminf(inv_e, 1.0f);
    float lr[NTL][2];
#pragma unroll
    for (int j = 0; j < NTL; ++j) {
      split(lsum[j], lr[j][0], lr[j][1]);
      lr[j][0] = column_sum(lr[j][0]);
      lr[j][1] = column_sum(lr[j][1]);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float l[2];
        split(lv[j][b], l[0], l[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          l[c] = column_sum(l[c]);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            acc[j][b][m][c] = fmaf(acc[j][b][m][c] * unit_e, unit_v, l[c]);
            acc[j][b][m][2 + c] = fmaf(acc[j][b][m][2 + c] * (unit_e * 0.0625f), unit_v, l[c]);
          }
        }
      }
    }
    // ---- warps joined, always in the same order: the upper half hands its sums to the lower half, whose sums then lie
    // side by side for all threads to add
    const bool small = s.re < (1 << 30);  // 32-bit division where it will do
    const int c_first = small ? static_cast<uint32_t>(s.rb) / static_cast<uint32_t>(share) : static_cast<int>(s.rb / share);
    const int c_last =
        small ? static_cast<uint32_t>(s.re - 1) / static_cast<uint32_t>(share) : static_cast<int>((s.re - 1) / share);
    const size_t slot = static_cast<size_t>(blockIdx.x) + s.row;
    const Seg done = s;
    float *joined = reinterpret_cast<float *>(smem + C::OFF_JOIN);      // [slot][column][kColStride]
    float *jml = joined + C::kSlots * C::N * C::kColStride;             // [slot][column] maximum, sum
    if (!C::kApart) __syncthreads();  // the ring is idle
    float *mine = joined + static_cast<size_t>(pw < C::kSlots ? pw : pw - C::kSlots) * C::N * C::kColStride;
    float *mml = jml + (pw < C::kSlots ? pw : pw - C::kSlots) * C::N * 2;
    auto put = [&]() {
#pragma unroll
      for (int j = 0; j < NTL; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = (cg * NTL + j) * 8 + 2 * t + c;
          if (g == 0) *reinterpret_cast<float2 *>(mml + col * 2) = make_float2(mref[j][c], lr[j][c]);
          float *o = mine + col * C::kColStride + g * 8;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            *reinterpret_cast<float4 *>(o + b * 64) =
                make_float4(acc[j][b][0][c], acc[j][b][0][2 + c], acc[j][b][1][c], acc[j][b][1][2 + c]);
            *reinterpret_cast<float4 *>(o + b * 64 + 4) =
                make_float4(acc[j][b][2][c], acc[j][b][2][2 + c], acc[j][b][3][c], acc[j][b][3][2 + c]);
          }
        }
    };
    if (pw >= C::kSlots) put();
    __syncthreads();
    if (more) {
      x += s.p1 - s.p0;
      s = s_seg;
      load_queries();
      open_part();  // the next part's ids, and below its first copies, come in beside the joins
    }
    if (pw < C::kSlots) {
      if (pw + C::kSlots < C::PW) {
#pragma unroll
        for (int j = 0; j < NTL; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = (cg * NTL + j) * 8 + 2 * t + c;
            const float2 o = *reinterpret_cast<const float2 *>(mml + col * 2);
            const float m = fmaxf(mref[j][c], o.x), fa = fast_exp2(mref[j][c] - m), fb = fast_exp2(o.x - m);
            mref[j][c] = m;
            lr[j][c] = fmaf(lr[j][c], fa, o.y * fb);
            const float *v = mine + col * C::kColStride + g * 8;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                acc[j][b][z][c] = fmaf(acc[j][b][z][c], fa, v[b * 64 + 2 * z] * fb);
                acc[j][b][z][2 + c] = fmaf(acc[j][b][z][2 + c], fa, v[b * 64 + 2 * z + 1] * fb);
              }
          }
        __syncwarp();
      }
      put();
    }
    if (more) {
      classify();
      if (C::kApart && !dead) issue();
    }
    __syncthreads();
    // ---- the row's result, or a record of its part
    for (int i = tid; i < M * (D / 8); i += C::kThreads) {
      const int col = i / (D / 8), d0 = (i - col * (D / 8)) * 8;
      float m = kNoMax, l = 0.0f, v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < C::kSlots; ++w) m = fmaxf(m, jml[(w * C::N + col) * 2]);
#pragma unroll
      for (int w = 0; w < C::kSlots; ++w) {
        const float f = fast_exp2(jml[(w * C::N + col) * 2] - m);
        l = fmaf(jml[(w * C::N + col) * 2 + 1], f, l);
        const float *o = joined + (w * C::N + col) * C::kColStride + d0;
        const float4 a = *reinterpret_cast<const float4 *>(o), b = *reinterpret_cast<const float4 *>(o + 4);
        v[0] = fmaf(a.x, f, v[0]), v[1] = fmaf(a.y, f, v[1]), v[2] = fmaf(a.z, f, v[2]), v[3] = fmaf(a.w, f, v[3]);
        v[4] = fmaf(b.x, f, v[4]), v[5] = fmaf(b.y, f, v[5]), v[6] = fmaf(b.z, f, v[6]), v[7] = fmaf(b.w, f, v[7]);
      }
      if (c_first == c_last) {
        const int qi = col / G;
        const size_t o = static_cast<size_t>(done.qoff + qi) * p.hq + done.h * G + (col - qi * G);
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
        for (int z = 0; z < 8; ++z) v[z] *= inv;
        *reinterpret_cast<uint4 *>(p.out + o * D + d0) = Vec16<__nv_bfloat16>::pack(v);
        if (d0 == 0) {
          p.lse[o] = l != 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
          if (kView && l == 0.0f) set_error(p.err, kErrLength);
        }
      } else {
        float *rec = p.part + (slot * p.ncol + col) * D + d0;
        __stcg(reinterpret_cast<float4 *>(rec), make_float4(v[0], v[1], v[2], v[3]));
        __stcg(reinterpret_cast<float4 *>(rec + 4), make_float4(v[4], v[5], v[6], v[7]));
        if (d0 == 0) __stcg(&p.ml[slot * p.ncol + col], make_float2(m, l));
      }
    }
    if (c_first != c_last) {
      __syncthreads();
      if (tid == 0) {
        const int parts = c_last - c_first + 1;
        const int old = atom_add_acq_rel_gpu(&p.counters[c_first], 1);
        s_flag = old == parts - 1;
        if (s_flag) p.counters[c_first] = 0;  // left at zero for the next call
      }
      __syncthreads();
      if (s_flag) {
        // part k of the row lies in slot c_first + k + row; weights first, then every thread sums its values in order
        const int parts = c_last - c_first + 1;
        const size_t slot0 = static_cast<size_t>(c_first) + done.row;
        float *w = joined;  // [parts][M] weights over the row's sum
        float2 *mls = reinterpret_cast<float2 *>(joined);
        // the maxima and sums come in as pairs; a column's thread turns them into weights in place (first half of a pair)
        for (int i = tid; i < parts * M; i += C::kThreads) {
          const int k = i / M, col = i - k * M;
          mls[i] = __ldcg(&p.ml[(slot0 + k) * p.ncol + col]);
        }
        __syncthreads();
        for (int col = tid; col < M; col += C::kThreads) {
          float m = kNoMax, l = 0.0f;
          for (int k = 0; k < parts; ++k) m = fmaxf(m, mls[k * M + col].x);
          for (int k = 0; k < parts; ++k) {
            const float2 z = mls[k * M + col];
            const float f = fast_exp2(z.x - m);
            l = fmaf(z.y, f, l);
            w[2 * (k * M + col)] = f;
          }
          const int i = col / G;
          p.lse[static_cast<size_t>(done.qoff + i) * p.hq + done.h * G + (col - i * G)] =
              l != 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
          if (kView && l == 0.0f) set_error(p.err, kErrLength);
          w[2 * col + 1] = l != 0.0f ? 1.0f / l : 0.0f;  // of part 0's pair: the factor of the whole column
        }
        __syncthreads();
        for (int i = tid; i < M * (D / 8); i += C::kThreads) {
          const int col = i / (D / 8), d0 = (i - col * (D / 8)) * 8;
          float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
          for (int k = 0; k < parts; ++k) {
            const float *rec = p.part + ((slot0 + k) * p.ncol + col) * D + d0;
            const float4 a = __ldcg(reinterpret_cast<const float4 *>(rec));
            const float4 b = __ldcg(reinterpret_cast<const float4 *>(rec + 4));
            const float f = w[2 * (k * M + col)];
            v[0] = fmaf(a.x, f, v[0]), v[1] = fmaf(a.y, f, v[1]), v[2] = fmaf(a.z, f, v[2]), v[3] = fmaf(a.w, f, v[3]);
            v[4] = fmaf(b.x, f, v[4]), v[5] = fmaf(b.y, f, v[5]), v[6] = fmaf(b.z, f, v[6]), v[7] = fmaf(b.w, f, v[7]);
          }
          const float inv = w[2 * col + 1];
#pragma unroll
          for (int z = 0; z < 8; ++z) v[z] *= inv;
          const int qi = col / G;
          const size_t o = static_cast<size_t>(done.qoff + qi) * p.hq + done.h * G + (col - qi * G);
          *reinterpret_cast<uint4 *>(p.out + o * D + d0) = Vec16<__nv_bfloat16>::pack(v);
        }
      }
    }
    if (!more) break;
    if (!C::kApart) fence_proxy_async_smem();  // the next copies write the memory that the joins used
    __syncthreads();
    if (!C::kApart && !dead) issue();
  }
}

template <int D, int NTL, int CS, bool kView>
cudaError_t launch(const AParams &p, cudaStream_t s) {
  using C = Cfg<D, NTL, CS>;
  static_assert(C::kMaxGrid <= kMaxCtas, "record slots");
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev & 63]) {
    e = cudaFuncSetAttribute(attn_kernel<D, NTL, CS, kView>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != cudaSuccess) return e;
    ready[dev & 63] = true;
  }
  // Rows of up to 16 pages a warp get a CTA each, which needs no scan, records, atomic or merge; longer ones are shared
  // out. Both sides on a GB300, proposals over 32, 256 and 2400 rows, us by row / shared out: 60 pages 10 / 15, 17 / 26,
  // 114 / 126; 120 pages 16 / 17, 25 / 30, 161 / 175 (110 pages); 150 pages over 32 rows 18 / 16. Windows of 16, 32 and 64
  // columns over 8, 32 and 256 rows: 30 pages 9.4 / 18, 16 / 27, 24 / 38; 9.8 / 19, 16 / 28, 24 / 40; 19 / 28, 31 / 43,
  // 48 / 58; 60 pages over 32 rows 13 / 21, 22 / 31, 36 / 37; 120 pages (64 for two groups of warps) over 32 rows 19 / 22, 34 /
  // 31, over 256 rows 39 / 43, 70 / 77. The rule goes by the table's width, which the host knows, not by the lengths: short
  // rows in a wider table are shared out.
  AParams q = p;
  const int grid = std::min(device_sm_count() * C::kCtas, C::kMaxGrid);
  const int64_t rows = static_cast<int64_t>(p.R) * p.hkv;
  q.by_row = (kView ? p.view.cap : p.max_pages) <= 16 * C::PW && rows <= 0x7fffffff;
  return launch_pdl(attn_kernel<D, NTL, CS, kView>, dim3(q.by_row ? static_cast<int>(rows) : grid), dim3(C::kThreads),
                    C::BYTES, s, q);
}

// Column tiles of 8: up to 4 a warp; wider windows go to two groups of warps that read the same pages.
template <int D, bool kView>
cudaError_t launch_tiles(const AParams &p, cudaStream_t s) {
  const int tiles = (p.ncol + 7) / 8;
  if (kView || tiles == 1) return launch<D, 1, 1, kView>(p, s);
  if (tiles == 2) return launch<D, 2, 1, false>(p, s);
  if (tiles == 3) return launch<D, 3, 1, false>(p, s);
  if (tiles == 4) return launch<D, 4, 1, false>(p, s);
  if (tiles <= 6) return launch<D, 3, 2, false>(p, s);
  return launch<D, 4, 2, false>(p, s);
}


AParams params(const PackedArgs &pa, const MapArgs &m, const void *q, void *out, float *lse, void *ws, int ncol,
               int *err) {
  AParams p{};
  p.k = static_cast<const __nv_bfloat16 *>(pa.pool.k);
  p.v = static_cast<const __nv_bfloat16 *>(pa.pool.v);
  p.packed = static_cast<const unsigned char *>(pa.packed);
  p.P16 = pa.pool.num_pages;
  p.P4 = pa.num_packed;
  p.hkv = pa.pool.hkv;
  p.hq = pa.pool.hq;
  p.R = m.R;
  p.bt = m.bt;
  p.max_pages = m.max_pages;
  p.ctx_len = m.ctx_len;
  p.seq_len = m.seq_len;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.ncol = ncol;
  p.err = err;
  const size_t rows = static_cast<size_t>(m.R) * p.hkv, slots = rows + kMaxCtas;
  unsigned char *w = static_cast<unsigned char *>(ws);
  p.counters = reinterpret_cast<int *>(w);
  w += kCounterBytes;
  p.ml = reinterpret_cast<float2 *>(w);
  w += (slots * ncol * 8 + 255) / 256 * 256;
  p.part = reinterpret_cast<float *>(w);
  return p;
}

}  // namespace

size_t packed_workspace_bytes(int R, int hkv, int hq, int d, int max_q) {
  const size_t rows = static_cast<size_t>(R) * hkv, slots = rows + kMaxCtas;
  const size_t ncol = static_cast<size_t>(hq / hkv) * max_q;
  return kCounterBytes + (slots * ncol * 8 + 255) / 256 * 256 + slots * ncol * d * 4;
}

cudaError_t launch_propose_packed(const PackedArgs &pa, const MapArgs &m, const ViewArgs &v, const void *q, void *out,
                                  float *lse, void *ws, int *err, cudaStream_t s) {
  AParams p = params(pa, m, q, out, lse, ws, pa.pool.hq / pa.pool.hkv, err);
  p.view = v;
  p.max_q = 1;
  p.total_q = m.R;
  return pa.pool.d == 128 ? launch_tiles<128, true>(p, s) : launch_tiles<64, true>(p, s);
}

cudaError_t launch_verify_packed(const PackedArgs &pa, const MapArgs &m, int max_q, int total_q,
                                 const int32_t *q_offsets, const int32_t *q_start, const void *q, void *out,
                                 float *lse, void *ws, int *err, cudaStream_t s) {
  AParams p = params(pa, m, q, out, lse, ws, pa.pool.hq / pa.pool.hkv * max_q, err);
  p.q_offsets = q_offsets;
  p.q_start = q_start;
  p.max_q = max_q;
  p.total_q = total_q;
  return pa.pool.d == 128 ? launch_tiles<128, false>(p, s) : launch_tiles<64, false>(p, s);
}

}  // namespace kap
