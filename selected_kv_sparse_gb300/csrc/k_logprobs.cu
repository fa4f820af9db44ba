// k_logprobs.cu - log probabilities of given tokens, entropy, rank and the best alternatives (sm_103a).
//
// Mathematics, in base 2 (c = log2 e): with a reference M, y_i = x_i c - M, S = sum 2^y_i and T = sum 2^y_i y_i,
//   log p_t = ln 2 (y_t - log2 S),   entropy = ln 2 (log2 S - T / S).
// M is a number of its own (the rounded product of a maximum and c), so y_i has one rounding and partial sums of
// different references join by powers of two. Logits below -1e7 are lifted there on the way in: their 2^y is 0 all the
// same and the entropy's 0 * y stays 0 for -infinity. Rows whose maximum lies outside (-9e5, 1e6), where that would
// distort or M's own rounding would leave a large y, are summed again from x - max.
// Rank: tokens before the given one count with >= on the pieces of the row that lie before it and with > behind it.
// Alternatives: the row is cut into at most 256 tiles whose maxima are kept. A token among the first n of the order lies
// in one of the first n tiles by (maximum, position): every tile before its own holds a token that comes before it. So
// only those n tiles are read again (from L2), and the n-th tile's maximum bars nearly all of their tokens.
//
// Bound by HBM: one pass over the logits; at bf16 the exponential unit (16 a cycle and SM) would allow 1.36 times the
// measured copy rate, so the loop keeps to packed bf16 compares and maxima and to pairs of fp32. A warp streams
// chunks of 512 logits with the next chunk's loads in flight and its own running sums: no barriers. Rows that are
// too few to fill the GPU are split over CTAs; the last one to finish a row joins the parts in their order.
// On a GB300, vocabulary 128256: 2048 rows of bf16 with 20 alternatives 118 us, 4.4 TB/s, 66% of the measured copy rate (101
// us without alternatives): 10 instructions a logit fill 68% of the issue slots, the rest are waits; of fp32 177 us, 87%; 20
// rows of fp32 with 5 alternatives 9.6 us. 200 and 400 rows of bf16 take 22 and 35 us (2.3 to 2.9 times the copy rate's time:
// the CTAs come to 1.3 waves), 511 rows 42, 512 rows 39. Where a row has fewer tiles than alternatives (below 16384 tokens
// for 32) every token is a candidate: 4096 rows of 4000 take 31 us without and 187 us with 20 alternatives.
#include "kap_device.cuh"
#include "kap_launch.h"

#include <algorithm>

namespace kap {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kChunk = 512;              // logits of a warp's step, 16 a lane
constexpr int kMaxTiles = kLpThreads;    // tiles of a row whose maxima are kept: one a thread
constexpr int kMaxSplit = 32;            // CTAs of a row
constexpr int kSplitRows = 512;          // from here on there is a CTA a row
constexpr size_t kCounterBytes = kSplitRows * sizeof(int);  // whatever the rows: calls of any sizes may take one
                                                            // workspace in turn
constexpr float kC = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -1e7f;         // logits are lifted to it
constexpr float kNoRef = -1e6f;          // reference before any logit: above what is lifted
constexpr float kSlack = 10.0f;          // how far a logit may exceed a lane's reference

struct LParams {
  const void *logits;
  int V, rows, top_n, split, tile_chunks;  // a tile is tile_chunks chunks
  int64_t stride;
  const int32_t *tokens;
  float *lp, *ent;
  int32_t *rank, *top_ids;
  float *top_lp;
  int *counters;
  float4 *parts;    // [row][kMaxSplit]: maximum, reference sum S, T, tokens before (bits)
  float *tops;      // [row][kMaxTiles] maxima of the tiles' numbers
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Maximum of a warp's numbers; NaN when there is none.
__device__ __forceinline__ float warp_top(float a) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ unsigned long long rank_key(uint32_t k, int t) {
  return (static_cast<unsigned long long>(k) << 32) | (0xffffffffu - static_cast<uint32_t>(t));
}
__device__ __forceinline__ float key_value(uint32_t k) {  // inverse of order_key
  return k == 0u ? NAN : __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// M of one reference less M of another, from above -1e30: also where both overflow (such rows are summed again).
__device__ __forceinline__ float shift(float from, float to) {
  return fmaxf(__fmul_rn(from, kC) - __fmul_rn(to, kC), -1e30f);
}

// Running sums of a lane: true maximum, reference (a logit), S and T.
struct Sums {
  float mx = -INFINITY, ref = kNoRef, s = 0.0f, t = 0.0f;
};
// b joined to a: sums over the larger reference.
__device__ __forceinline__ void join(Sums &a, const Sums &b) {
  a.mx = fmaxf(a.mx, b.mx);
  const float r = fmaxf(a.ref, b.ref);
  const float da = shift(a.ref, r), db = shift(b.ref, r);
  const float fa = exp2_fast(da), fb = exp2_fast(db);
  a.t = fmaf(fa, a.t, a.s * fa * da) + fmaf(fb, b.t, b.s * fb * db);
  a.s = fmaf(fa, a.s, fb * b.s);
  a.ref = r;
}

// 16 logits of a lane: VEC 16-byte loads of EPV logits, vector (j * 32 + lane) of the chunk.
template <class T>
struct Lane16 {
  static constexpr int EPV = Vec16<T>::N, VEC = 16 / EPV;
  uint4 v[VEC];
  __device__ __forceinline__ void load(const T *chunk, int lane) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const T *a = chunk + (j * 32 + lane) * EPV;
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[j].x), "=r"(v[j].y), "=r"(v[j].z), "=r"(v[j].w)
                   : "l"(a));
    }
  }
  // position in the chunk of value i
  __device__ __forceinline__ static int at(int i, int lane) { return ((i / EPV) * 32 + lane) * EPV + i % EPV; }
  __device__ __forceinline__ void values(float *x) const {
#pragma unroll
    for (int j = 0; j < VEC; ++j) Vec16<T>::unpack(v[j], x + j * EPV);
  }
};

// A lane's running sums over its chunks: S and T as pairs.
struct Run {
  float mx = -INFINITY, ref = kNoRef;
  F2 s = f2(0.0f, 0.0f), t = f2(0.0f, 0.0f);
  __device__ __forceinline__ void lift(float m) {  // raises the reference to a new chunk's maximum where it must
    float a, b;
    split(s, a, b);
    if (m > ref + kSlack || (a == 0.0f && m > ref)) {
      const float d = shift(ref, m), f = exp2_fast(d);
      const F2 ff = f2(f, f);
      t = fma2(t, ff, mul2(s, f2(f * d, f * d)));  // sum 2^(y + d) (y + d)
      s = mul2(s, ff);
      ref = m;
    }
  }
  __device__ __forceinline__ Sums sums() const {
    Sums u;
    float a, b;
    u.mx = mx;
    u.ref = ref;
    split(s, a, b);
    u.s = a + b;
    split(t, a, b);
    u.t = a + b;
    return u;
  }
};
// Logits before the given one, counted for two halves of a word: minus a half's count in either half, the lower one's
// borrow taken from the upper (a warp has 2^24 / 4096 chunks at most, 8 a half each).
__device__ __forceinline__ int halves(uint32_t acc) {
  const uint32_t lo = (0u - acc) & 0xffffu, d = (acc + lo) >> 16;
  return static_cast<int>(lo + ((lo - d) & 0xffffu));
}

// Two logits into the running pairs of S and T.
__device__ __forceinline__ void add_pair(F2 x, F2 c, F2 m, F2 &s, F2 &t) {
  const F2 y = fma2(x, c, m);
  float a, b;
  split(y, a, b);
  const F2 e = f2(exp2_fast(a), exp2_fast(b));
  s = add2(s, e);
  t = fma2(e, y, t);
}
// A whole chunk: maximum, sums, and how many logits are above xt (or at least xt when `ge`).
__device__ __forceinline__ float chunk_pass(const Lane16<float> &c, Run &u, float xt, bool ge, int &before, uint32_t &) {
  float x[16];
  c.values(x);
  float m = x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) m = fmaxf(m, x[i]);
  u.lift(m);
  const float M = u.ref * kC;
  if (ge) {
#pragma unroll
    for (int i = 0; i < 16; ++i) before += x[i] >= xt ? 1 : 0;
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) before += x[i] > xt ? 1 : 0;
  }
  const F2 cc = f2(kC, kC), mm = f2(-M, -M);
#pragma unroll
  for (int i = 0; i < 16; i += 2) add_pair(f2(max_nan(x[i], kLowest), max_nan(x[i + 1], kLowest)), cc, mm, u.s, u.t);
  return m;
}
__device__ __forceinline__ float chunk_pass(const Lane16<__nv_bfloat16> &c, Run &u, float xt, bool ge, int &,
                                            uint32_t &acc) {
  const uint32_t w[8] = {c.v[0].x, c.v[0].y, c.v[0].z, c.v[0].w, c.v[1].x, c.v[1].y, c.v[1].z, c.v[1].w};
  __nv_bfloat162 h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
  const __nv_bfloat162 m2 = __hmax2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])),
                                    __hmax2(__hmax2(h[4], h[5]), __hmax2(h[6], h[7])));
  const float m = fmaxf(__low2float(m2), __high2float(m2));
  u.lift(m);
  const float M = u.ref * kC;
  const __nv_bfloat162 t2 = __float2bfloat162_rn(xt), low = __float2bfloat162_rn(kLowest);  // xt is a bf16
  if (ge) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc += __hge2_mask(h[i], t2);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc += __hgt2_mask(h[i], t2);
  }
  const F2 cc = f2(kC, kC), mm = f2(-M, -M);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 l = __hmax2_nan(h[i], low);
    const uint32_t b = *reinterpret_cast<const uint32_t *>(&l);
    add_pair(f2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)), cc, mm, u.s, u.t);
  }
  return m;
}

// Bits of the lane's values that are at least b, in one word, and the value that a bit stands for. For bf16, b is above a
// bf16 number by less than one place (its low bits are those that a key loses), so its upper half compares alike.
__device__ __forceinline__ unsigned reach(const Lane16<float> &c, float b) {
  float x[16];
  c.values(x);
  unsigned hit = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) hit |= x[i] >= b ? 1u << i : 0u;
  return hit;
}
__device__ __forceinline__ unsigned reach(const Lane16<__nv_bfloat16> &c, float b) {
  const uint32_t w[8] = {c.v[0].x, c.v[0].y, c.v[0].z, c.v[0].w, c.v[1].x, c.v[1].y, c.v[1].z, c.v[1].w};
  const uint32_t u = __float_as_uint(b) >> 16, uu = u | (u << 16);
  const __nv_bfloat162 b2 = *reinterpret_cast<const __nv_bfloat162 *>(&uu);
  unsigned hit = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    hit |= __hge2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), b2) & (0x00010001u << i);
  return hit;
}
template <class T>
__device__ __forceinline__ int bit_of(int i) { return sizeof(T) == 2 ? (i >> 1) + (i & 1) * 16 : i; }
template <class T>
__device__ __forceinline__ int value_of(int bit) { return sizeof(T) == 2 ? (bit & 15) * 2 + (bit >> 4) : bit; }

// Keys of a warp in descending order (bitonic).
template <class K>
__device__ __forceinline__ K warp_sort_desc(K k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d >= 1; d >>= 1) {
      const K o = __shfl_xor_sync(0xffffffffu, k, d);
      const bool keep_max = ((lane & d) == 0) == ((lane & size) == 0);
      k = keep_max ? (o > k ? o : k) : (o > k ? k : o);
    }
  return k;
}
// The 32 largest of two descending lists, descending: a, and b given backwards.
__device__ __forceinline__ uint32_t warp_merge_desc(uint32_t a, uint32_t b_backwards, int lane) {
  uint32_t k = max(a, b_backwards);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const uint32_t o = __shfl_xor_sync(0xffffffffu, k, d);
    k = (lane & d) == 0 ? max(k, o) : min(k, o);
  }
  return k;
}
// How many keys of the block's sorted warps (32 a warp, descending, distinct or 0) come before k, the lane-th of its own.
template <class K>
__device__ __forceinline__ int block_rank(const K *lists, K k, int warp, int lane) {
  int r = lane;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
    if (w == warp) continue;
    int n = 0;
#pragma unroll
    for (int step = 16; step >= 1; step >>= 1) n += lists[w * 32 + n + step - 1] > k ? step : 0;
    n += lists[w * 32 + n] > k ? 1 : 0;
    r += n;
  }
  return r;
}

// A chunk one by one: the given token's, a row's ends, rows whose token is a NaN. Sums s, t of the lane go on from u's.
// A call of its own: in the loop it takes registers from the chunks that count (2048 rows 124 us against 119).
struct Single {
  float m, ref, s, t;
  int before;
};
template <class T>
__device__ __noinline__ Single single_chunk(const T *base, int c, int lane, int off, int end, int tpos, float xt, Sums u) {
  const uint32_t kt = order_key(xt);
  float v[16];
  bool in[16];
  Single z{NAN, u.ref, u.s, u.t, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int pos = c * kChunk + Lane16<T>::at(i, lane);
    in[i] = pos >= off && pos < end;
    v[i] = in[i] ? to_f(base[pos]) : NAN;
    z.m = fmaxf(z.m, v[i]);
    if (in[i] && tpos >= 0) {
      const uint32_t k = order_key(v[i]);
      z.before += k > kt || (k == kt && pos < tpos) ? 1 : 0;
    }
  }
  if (z.m > z.ref + kSlack || (z.s == 0.0f && z.m > z.ref)) {
    const float d = shift(z.ref, z.m), f = exp2_fast(d);
    z.t = fmaf(z.t, f, z.s * f * d);
    z.s *= f;
    z.ref = z.m;
  }
  const float M = z.ref * kC;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (!in[i]) continue;
    const float y = fmaf(max_nan(v[i], kLowest), kC, -M);
    const float e = exp2_fast(y);
    z.s += e;
    z.t = fmaf(e, y, z.t);
  }
  return z;
}

template <class T>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_kernel(const LParams p) {
  __shared__ Sums s_sums[kLpWarps];
  __shared__ int s_before[kLpWarps], s_last;
  __shared__ float s_top[kMaxTiles];
  __shared__ int s_tile[kMaxTiles], s_ntile, s_ncand;
  __shared__ uint32_t s_sorted[kMaxTiles], s_bar;
  __shared__ unsigned long long s_list[kLpThreads];
  __shared__ float s_ref, s_logz;
  __shared__ int s_kind;
  grid_dependency_sync();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.split, part = blockIdx.x - row * p.split;
  const T *x = static_cast<const T *>(p.logits) + row * p.stride;
  // positions are counted from the 16-byte boundary at or before the row: `off` of them lie before it
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const T *base = x - off;
  const int end = off + p.V;
  const int chunks = (end + kChunk - 1) / kChunk, tiles = (chunks + p.tile_chunks - 1) / p.tile_chunks;
  const int tok = p.tokens[row];
  const bool has = tok >= 0 && tok < p.V;
  const int tpos = off + tok;
  float *tops = p.split > 1 ? p.tops + static_cast<size_t>(row) * kMaxTiles : s_top;

  // ---- this warp's tiles: every (split * warps)-th
  Run run;
  int before = 0;
  uint32_t acc = 0u;
  const int w0 = part * kLpWarps + warp, ws = p.split * kLpWarps;
  // chunks [c_lo, c_hi) lie inside the row; the chunk of the given token is apart, and so is a row whose token is a NaN
  const int c_lo = off ? 1 : 0, c_hi = end / kChunk;
  auto whole = [&](int c) { return c >= c_lo && c < c_hi; };
  const int c_tok = has ? tpos / kChunk : -1;
  float xt = 0.0f;
  Lane16<T> cur, nxt;
  int tile = w0, c = tile * p.tile_chunks;
  if (tile < tiles && whole(c)) cur.load(base + c * kChunk, lane);
  if (has) xt = to_f(x[tok]);
  const bool odd = xt != xt;
  float tmax = NAN;  // maximum of the tile's numbers
  while (tile < tiles) {
    // the next chunk: of this tile, or of the warp's next one
    int nc = c + 1, nt = tile;
    if (nc == (tile + 1) * p.tile_chunks || nc >= chunks) nt = tile + ws, nc = nt * p.tile_chunks;
    if (whole(nc)) nxt.load(base + nc * kChunk, lane);
    float m;
    if (whole(c) && c != c_tok && !odd) {
      m = chunk_pass(cur, run, xt, c < c_tok, before, acc);
    } else {
      const Single z = single_chunk(base, c, lane, off, end, has ? tpos : -1, xt, run.sums());
      m = z.m;
      before += z.before;
      run.ref = z.ref;
      run.s = f2(z.s, 0.0f);
      run.t = f2(z.t, 0.0f);
    }
    tmax = fmaxf(tmax, m);
    if (nt != tile) {
      run.mx = fmaxf(run.mx, tmax);
      if (p.top_n > 0) {
        const float k = warp_top(tmax);
        if (lane == 0) tops[tile] = k;
      }
      tmax = NAN;
    }
    cur = nxt;
    tile = nt;
    c = nc;
  }
  Sums u = run.sums();
  before += halves(acc);
  // ---- lanes, then warps, joined in a fixed order
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    Sums b;
    b.mx = __shfl_xor_sync(0xffffffffu, u.mx, o);
    b.ref = __shfl_xor_sync(0xffffffffu, u.ref, o);
    b.s = __shfl_xor_sync(0xffffffffu, u.s, o);
    b.t = __shfl_xor_sync(0xffffffffu, u.t, o);
    join(u, b);
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) {
    s_sums[warp] = u;
    s_before[warp] = before;
  }
  __syncthreads();
  if (p.split > 1) {
    if (tid == 0) {
      for (int w = 1; w < kLpWarps; ++w) {
        join(u, s_sums[w]);
        before += s_before[w];
      }
      p.parts[static_cast<size_t>(row) * kMaxSplit * 2 + part * 2] = make_float4(u.mx, u.ref, u.s, u.t);
      p.parts[static_cast<size_t>(row) * kMaxSplit * 2 + part * 2 + 1] = make_float4(__int_as_float(before), 0, 0, 0);
      int old;
      asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p.counters + row), "r"(1) : "memory");
      s_last = old == p.split - 1;
      if (s_last) p.counters[row] = 0;  // left at zero for the next call
    }
    __syncthreads();
    if (!s_last) return;
    for (int i = tid; i < tiles; i += kLpThreads) s_top[i] = __ldcg(tops + i);
  }
  // ---- the row's sums
  if (warp == 0) {
    Sums r;
    int b = 0;
    const int n = p.split > 1 ? p.split : kLpWarps;
    if (p.split > 1) {
      float4 q = make_float4(-INFINITY, kNoRef, 0.0f, 0.0f);
      if (lane < n) {
        q = __ldcg(&p.parts[static_cast<size_t>(row) * kMaxSplit * 2 + lane * 2]);
        b = __float_as_int(__ldcg(&p.parts[static_cast<size_t>(row) * kMaxSplit * 2 + lane * 2 + 1].x));
      }
      r.mx = q.x, r.ref = q.y, r.s = q.z, r.t = q.w;
    } else if (lane < n) {
      r = s_sums[lane];
      b = s_before[lane];
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      Sums q;
      q.mx = __shfl_xor_sync(0xffffffffu, r.mx, o);
      q.ref = __shfl_xor_sync(0xffffffffu, r.ref, o);
      q.s = __shfl_xor_sync(0xffffffffu, r.s, o);
      q.t = __shfl_xor_sync(0xffffffffu, r.t, o);
      join(r, q);
    }
    b = __reduce_add_sync(0xffffffffu, b);
    if (lane == 0) {
      // kind 0: sums hold; 1: no distribution (NaN, an infinity on top, nothing left); 2: sum again from x - max
      int kind = 0;
      if (r.mx == INFINITY || r.mx == -INFINITY) kind = 1;
      else if (!(r.mx > -9e5f && r.mx < 1e6f)) kind = 2;  // which looks for NaN itself
      else if (r.s != r.s) kind = 1;
      s_kind = kind;
      // log p = (x - ref) - (log S of the terms over ref): no product that a far logit overflows
      const float l2 = log2f(r.s), res = fmaf(r.ref, kC, -__fmul_rn(r.ref, kC));
      s_ref = kind == 2 ? r.mx : r.ref;
      s_logz = (l2 - res) * kLn2;
      if (p.rank) p.rank[row] = has ? b : p.V;
      if (kind != 2) {
        p.lp[row] = !has ? -INFINITY : kind == 1 ? NAN : (xt - r.ref) - s_logz;
        if (p.ent) p.ent[row] = kind == 1 ? NAN : (l2 - r.t / r.s) * kLn2;
      }
    }
  }
  __syncthreads();
  if (s_kind == 2) {
    // far logits: sums of 2^((x - max) c), every term from the difference
    const float mx = s_ref;
    float a = 0.0f, b = 0.0f;
    bool bad = false;
    for (int t = tid; t < p.V; t += kLpThreads) {
      const float v = to_f(x[t]);
      bad |= v != v;
      const float d = fmaxf((v - mx) * kC, -1e30f), e = exp2_fast(d);
      a += e;
      b = fmaf(e, d, b);
    }
    if (bad) a = NAN;
    a = warp_sum(a);
    b = warp_sum(b);
    if (lane == 0) s_sums[warp].s = a, s_sums[warp].t = b;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kLpWarps; ++w) a += s_sums[w].s, b += s_sums[w].t;
      const float l2 = log2f(a);
      s_logz = l2 * kLn2;
      p.lp[row] = !has ? -INFINITY : (xt - mx) - s_logz;
      if (p.ent) p.ent[row] = (l2 - b / a) * kLn2;
    }
    __syncthreads();
  }
  if (p.top_n == 0) return;

  // ---- a bar that top_n tokens reach: the top_n-th of the tiles' maxima, without its low bits (which a bf16 does not
  // have), so that a maximum and its tile make one distinct word to sort. Tiles that reach it are read again.
  const int n = p.top_n;
  {
    uint32_t k = tid < tiles ? (order_key(s_top[tid]) & ~255u) | (255u - tid) : 0u;
    k = warp_sort_desc(k, lane);
    const int own = k != 0u ? 255 - static_cast<int>(k & 255u) : tiles == kMaxTiles ? 255 : tiles;
    s_sorted[tid] = k;
    if (tid == 0) s_ntile = 0, s_ncand = 0;
    __syncthreads();
    if (warp == 0) {  // the eight lists' 32 largest, pair by pair
      uint32_t a[kLpWarps / 2];
#pragma unroll
      for (int i = 0; i < kLpWarps / 2; ++i)
        a[i] = warp_merge_desc(s_sorted[2 * i * 32 + lane], s_sorted[(2 * i + 1) * 32 + 31 - lane], lane);
#pragma unroll
      for (int m = kLpWarps / 4; m >= 1; m >>= 1)
#pragma unroll
        for (int i = 0; i < m; ++i)
          a[i] = warp_merge_desc(a[i], __shfl_sync(0xffffffffu, a[i + m], 31 - lane), lane);
      if (lane == n - 1) s_bar = tiles >= n ? a[0] & ~255u : 0u;
    }
    __syncthreads();
    if (own < tiles && (k & ~255u) >= s_bar) s_tile[atomicAdd(&s_ntile, 1)] = own;
    __syncthreads();
  }
  const uint32_t bar = s_bar;
  const int nt = s_ntile;
  // ---- their tokens that reach the bar: hardly more than top_n where logits differ
  for (int z = warp; z < nt; z += kLpWarps) {
    const int c0 = s_tile[z] * p.tile_chunks, c1 = min(c0 + p.tile_chunks, chunks);
    for (int cc = c0; cc < c1; ++cc) {
      // above the key of -infinity the bar is a number and one compare decides; NaN counts only below it
      unsigned hit = 0u;
      if (whole(cc) && bar > 0x007fffffu) {
        cur.load(base + cc * kChunk, lane);
        hit = reach(cur, key_value(bar));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int pos = cc * kChunk + Lane16<T>::at(i, lane);
          const bool in = pos >= off && pos < end;
          hit |= in && order_key(to_f(base[in ? pos : off])) >= bar ? 1u << bit_of<T>(i) : 0u;
        }
      }
      while (hit) {
        const int i = value_of<T>(__ffs(hit) - 1), pos = cc * kChunk + Lane16<T>::at(i, lane);
        hit &= hit - 1;
        const int at = atomicAdd(&s_ncand, 1);
        if (at < kLpThreads) s_list[at] = rank_key(order_key(to_f(base[pos])), pos - off);
      }
    }
  }
  __syncthreads();
  unsigned long long k = 0ull;
  int r = lane;
  if (s_ncand <= 32) {  // one warp's sort is the order
    if (warp != 0) return;
    k = warp_sort_desc(lane < s_ncand ? s_list[lane] : 0ull, lane);
  } else {
    if (s_ncand <= kLpThreads) {
      k = warp_sort_desc(tid < s_ncand ? s_list[tid] : 0ull, lane);
      __syncthreads();
    } else {
      // many equal logits: every warp inserts its tiles' tokens into a sorted list of its own (lane i: its i-th)
      for (int z = warp; z < nt; z += kLpWarps) {
        const int p0 = s_tile[z] * p.tile_chunks * kChunk, p1 = min(p0 + p.tile_chunks * kChunk, chunks * kChunk);
        for (int pos = p0 + lane; pos < p1; pos += 32) {
          unsigned long long key = 0ull;
          if (pos >= off && pos < end) {
            const uint32_t u32 = order_key(to_f(base[pos]));
            if (u32 >= bar) key = rank_key(u32, pos - off);
          }
          unsigned long long worst = __shfl_sync(0xffffffffu, k, n - 1);
          unsigned m = __ballot_sync(0xffffffffu, key > worst);
          while (m) {
            const int src = __ffs(m) - 1;
            const unsigned long long q = __shfl_sync(0xffffffffu, key, src);
            const int at = __popc(__ballot_sync(0xffffffffu, k > q));
            const unsigned long long up = __shfl_up_sync(0xffffffffu, k, 1);
            k = lane < at ? k : lane == at ? q : up;
            worst = __shfl_sync(0xffffffffu, k, n - 1);
            m &= __ballot_sync(0xffffffffu, key > worst) & ~(1u << src);
          }
        }
      }
      __syncthreads();
    }
    s_list[tid] = k;
    __syncthreads();
    if (k != 0ull) r = block_rank(s_list, k, warp, lane);
  }
  if (k != 0ull && r < n) {
    const float v = key_value(static_cast<uint32_t>(k >> 32));
    const size_t o = static_cast<size_t>(row) * n + r;
    p.top_ids[o] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(k));
    p.top_lp[o] = s_kind == 1 ? NAN : (v - s_ref) - s_logz;
  }
}

// A row has at most V / kChunk + 2 chunks, wherever it starts in memory.
int tile_chunks_of(int V) { return (V / kChunk + 2 + kMaxTiles - 1) / kMaxTiles; }

}  // namespace

size_t logprobs_workspace_bytes(int rows, int vocab) {
  (void)vocab;
  const size_t n = static_cast<size_t>(std::min(rows, kSplitRows));
  return kCounterBytes + n * kMaxSplit * 32 + n * kMaxTiles * 4;
}

cudaError_t launch_logprobs(const void *logits, int dtype, int V, int64_t stride, int rows, const int32_t *tokens,
                            int top_n, float *lp, float *ent, int32_t *rank, int32_t *top_ids, float *top_lp, void *ws,
                            cudaStream_t s) {
  LParams p{};
  p.logits = logits;
  p.V = V;
  p.rows = rows;
  p.top_n = top_n;
  p.stride = stride;
  p.tokens = tokens;
  p.lp = lp;
  p.ent = ent;
  p.rank = rank;
  p.top_ids = top_ids;
  p.top_lp = top_lp;
  p.tile_chunks = tile_chunks_of(V);
  p.split = 1;
  if (rows < kSplitRows) {
    // about four CTAs an SM, each warp with one tile at least
    const int tiles = (V / kChunk + 1) / p.tile_chunks + 1;
    p.split = std::max(1, std::min({(4 * device_sm_count() + rows - 1) / rows, tiles / kLpWarps, kMaxSplit}));
  }
  const size_t n = static_cast<size_t>(std::min(rows, kSplitRows));
  unsigned char *w = static_cast<unsigned char *>(ws);
  p.counters = reinterpret_cast<int *>(w);
  w += kCounterBytes;
  p.parts = reinterpret_cast<float4 *>(w);
  w += n * kMaxSplit * 32;
  p.tops = reinterpret_cast<float *>(w);
  const int64_t grid = static_cast<int64_t>(rows) * p.split;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  if (dtype == 0)
    return launch_pdl(logprobs_kernel<__nv_bfloat16>, dim3(static_cast<unsigned>(grid)), dim3(kLpThreads), 0, s, p);
  return launch_pdl(logprobs_kernel<float>, dim3(static_cast<unsigned>(grid)), dim3(kLpThreads), 0, s, p);
}

}  // namespace kap
