// k_sample.cu - sampling of tokens with temperature, top-k, min-p and top-p from given random numbers (sm_103a).
//
// Mathematics, for a row of logits x with the largest m at temperature T: w_i = exp((x_i - m) / T). The rank order is
// logit descending, lower id first. The tokens among the first top_k that weigh min_p or more are a run of that order from
// its start, and so is the shortest part of it that holds top_p of its weight: what is kept is a least logit, all tokens
// above it and the first few ids of those at it. The token drawn is the first in id order at which the running sum of the
// kept weights passes u times their sum.
// Weights are whole numbers, 2^-44 of the largest each (fewer bits past 2^18 tokens, so that sums stay below 2^62), so
// sums do not depend on their order. Each is right to 2^-37 of itself and a unit, so a border falls as it would in 64-bit
// floating point unless it lies that close.
//
// A row belongs to a cluster of CTAs, each with a slice of it; they add up their parts through one another's shared
// memory. One pass over it gives the maximum, the weight to about 2^-16, and the maxima of its tiles. Then, by what the row
// needs:
//   - few candidates decide it (small top_k, or a weight that few tokens hold): the logits above a bar that enough of the
//     lanes' maxima reach are gathered from their tiles in one CTA, sorted and drawn from there;
//   - 16-bit logits: they are counted by value, each value is weighed once, and the borders follow from running sums over
//     the values;
//   - fp32 logits under top_p: a histogram in 1/16 octaves of weight bounds the border from both ends; one pass weighs all
//     logits and counts those inside the bounds; the part that holds the border is gathered and sorted;
//   - else the interval of the border is cut by its bits, 2048 parts a pass, until a part is one logit.
// The last three end with the kept weight of each warp's range of ids, and the warps then halve the range that the draw
// falls into.
//
// Bound by instructions for flat rows: some 70 a logit that is weighed in line, 100 where it is called for, and for
// 16-bit counts an atomic each, of which a warp's fall into the same banks 3 to 4 times. (Two CTAs an SM leave 64
// registers, and draw_kept spills 300 to 360 bytes, outside its loops: 0.2% of the instructions that run.) In graphs:
// 2048 bf16 rows of 128256 under top_p 505 us (a third of them flat, 110 to 170 us each; the others 25 to 45), where
// reading them takes 77; 80 fp32 rows with settings of their own 115; 300 bf16 rows of 32000 without limits 47; 4 rows
// 20, most of it joins and one CTA's sort.
#include "kap_device.cuh"
#include "kap_launch.h"

#include <algorithm>

namespace kap {
namespace {

constexpr int kSaThreads = 512;
constexpr int kSaCtas = 2;         // CTAs of an SM: one's joins and draws run under the other's passes, and the rows of all
                                   // (80 MB of 16-bit logits) stay in L2 between their passes
constexpr int kSaWarps = kSaThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinsPerThread = kBins / kSaThreads;
constexpr float kBinsPerOctave = 16.0f;
constexpr int kMaxCluster = 16;
using u64 = unsigned long long;

struct SParams {
  const void *logits;
  int V, rows, qb;   // qb: bits of the weight 1
  int64_t stride;
  const float *u, *temp, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
  float *logprob;
  int32_t *kept;
};

// ---------------------------------------------------------------------------------------------------- clusters
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void *p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ u64 ld_remote64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_remote32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_remote32(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// ---------------------------------------------------------------------------------------------------- weights
__device__ __forceinline__ float key_value(uint32_t k) {  // inverse of order_key
  return k == 0u ? NAN : __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
// 2^(-j/64) for j < 64: as a sum of two fp32 and times 2^44, from the exponential series.
struct Powers {
  float2 f[64];
  u64 q[64];
};
constexpr double power_series(int j) {
  const double x = -0.69314718055994530942 * j / 64.0;
  double t = 1.0, s = 1.0;
  for (int n = 1; n < 30; ++n) {
    t *= x / n;
    s += t;
  }
  return s;
}
constexpr Powers make_powers() {
  Powers t{};
  for (int j = 0; j < 64; ++j) {
    const double v = power_series(j);
    t.f[j].x = static_cast<float>(v);
    t.f[j].y = static_cast<float>(v - static_cast<double>(t.f[j].x));
    t.q[j] = static_cast<u64>(v * 17592186044416.0 + 0.5);
  }
  return t;
}
__device__ const Powers kPowers = make_powers();

// exp((x - m) / T) as a whole number of 2^-qb, right to 2^-37 of itself and a unit, for x <= m that is no NaN:
// with y = (m - x) log2 e / T as a sum of two fp32, k the nearest whole number to 64 y and r = y - k / 64,
//   2^-y = 2^(-k/64) (1 - t + t^2/2 - t^3/6 + t^4/24),  t = r ln 2 <= 0.0055, t's leading term again as two fp32.
// Its largest error is that t's low part (up to 2^-31.2) counts in t but not in t^2/2: 2^-38.7 of the weight, to which the
// square's and the products' roundings add as much again.
// Every operation is rounded as written, so that the form in line and the one out of line give the same number.
__device__ __forceinline__ u64 weight_inline(float x, float m, float ch, float cl, int down, const Powers *tab) {
  auto add = [](float a, float b) { return __fadd_rn(a, b); };
  auto sub = [](float a, float b) { return __fsub_rn(a, b); };
  auto mul = [](float a, float b) { return __fmul_rn(a, b); };
  auto fma = [](float a, float b, float c) { return __fmaf_rn(a, b, c); };
  // m - x, exactly (two-sum)
  const float dh = sub(m, x), bb = sub(m, dh), dl = add(sub(m, add(dh, bb)), sub(bb, x));
  const float yh = mul(dh, ch);
  const float yl = add(fma(dh, ch, -yh), fma(dh, cl, mul(dl, ch)));
  // weights from 2^-45 on are nothing; up to here no shift below reaches 64 (56 and the 6 of 2^24 tokens). Not so for an
  // infinite distance
  const bool some = yh < 56.0f;
  constexpr float kLn2h = 0.693147182464599609375f, kLn2l = -1.904654323148236017e-9f;
  const float kf = fma(some ? yh : 0.0f, 64.0f, 12582912.0f);   // 1.5 * 2^23: the sum's low bits are the nearest whole number
  const int k = static_cast<int>(__float_as_uint(kf) - 0x4b400000u);
  const float r = fma(sub(kf, 12582912.0f), -0.015625f, yh);
  const float rh = add(r, yl), rl = add(sub(r, rh), yl);   // y's low part is up to 2^-20: it counts in the square, too
  const float th = mul(rh, kLn2h), tl = add(fma(rh, kLn2h, -th), fma(rh, kLn2l, mul(rl, kLn2h)));
  const float q = fma(mul(th, th), fma(th, fma(th, 0.0416666679f, -0.166666672f), 0.5f), -tl);
  const float2 f = tab->f[k & 63];
  const float ph = mul(f.x, -th);
  const float pl = add(fma(f.x, -th, -ph), fma(f.x, q, mul(f.y, -th)));
  // ph + pl in units of 2^-44, through the low bits of sums at 3 (unit 2^-22) and at 3 * 2^-22
  const float u = add(ph, pl), ub = sub(u, ph), ul = add(sub(ph, sub(u, ub)), sub(pl, ub));
  const float s1 = add(u, 3.0f);
  const int i1 = static_cast<int>(__float_as_uint(s1) - 0x40400000u);
  const float rest = add(sub(u, sub(s1, 3.0f)), ul);
  const int i2 = static_cast<int>(__float_as_uint(add(rest, 7.152557373046875e-7f)) - 0x35400000u);
  const u64 w = tab->q[k & 63] + static_cast<u64>(static_cast<int64_t>(i1) * (1 << 22) + i2);
  const int e = (k >> 6) + down;
  return some ? (w + ((u64(1) << e) >> 1)) >> e : u64(0);
}
// Out of line: passes that weigh logits in several places would not stay in the instruction cache.
__device__ __noinline__ u64 weight_of(float x, float m, float ch, float cl, int down, const Powers *tab) {
  return weight_inline(x, m, ch, cl, down, tab);
}
struct Weigh {
  float m, ch, cl;   // largest logit; log2 e / T
  int down;          // 44 - qb
  const Powers *tab;
  __device__ __forceinline__ u64 operator()(float x) const { return weight_of(x, m, ch, cl, down, tab); }
  __device__ __forceinline__ u64 here(float x) const { return weight_inline(x, m, ch, cl, down, tab); }   // passes over all
};

constexpr int kTiles = 64;         // tiles of a warp's range whose maxima are kept, two a lane
constexpr int kFew = 2 * kSaThreads;   // candidates that are sorted and drawn from directly
// top_k up to which the candidates are gathered. Gathered / not, bf16 rows of 128256 in graphs: top_k 200 4 rows 26 / 37 us,
// 80 rows 42 / 63, 2048 rows 462 / 652; top_k 400 42 / 37, 62 / 63 and 960 / 656 (fp32: 42 / 45, 70 / 86).
constexpr int kMaxFewK = 256;
// Candidates to gather, about, where top_k does not say. More of them decide more rows but take longer to sort: 4, 80 and
// 2048 bf16 rows under top_p, a third of them flat: 64 of them 47, 74 and 507 us; 32 46, 73 and 478; 128 47, 78 and 576;
// 256 50, 85 and 764.
constexpr int kFewBar = 64;
// Logits of 16 bits from 2^-10 to 2^10 in magnitude, counted by value: 2560 of either sign, by their bits.
constexpr int kValues = 5120, kHalfValues = kValues / 2;
constexpr uint32_t kFirstValue = 0x3A80, kEndValue = 0x4480;   // bits of 2^-10 and 2^10
constexpr int kOdd = 1024;         // logits of other magnitudes that a CTA keeps aside

struct Shared {
  uint32_t hist[kValues];
  union {
    u64 weight[kValues];   // of each counted value
    struct {
      u64 list[kFew], sorted[kFew], w[kFew];   // candidates: key and inverted id; their weights
    } few;
  };
  Powers powers;
  float odd[kOdd];
  u64 scan[kSaWarps], scan2[kSaWarps];   // of block-wide sums: who reads them ends with a barrier, so that the next may write
  u64 sums[3][2];   // values for the other CTAs, in turn: a slot is written again two exchanges later
  u64 pick[6];
  float fscan[kSaWarps];
  u64 own_w[kSaWarps], own_n[kSaWarps], cut;   // candidates above the border: weight, number, and at it, of each warp
  uint32_t few_count, few_done, odd_count;
  uint32_t joined[];   // [kValues] the cluster's histogram, where it has more than one CTA
};

__device__ __forceinline__ u64 shfl_up64(u64 v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_top(float a) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t add_remote32(uint32_t a, uint32_t v) {
  uint32_t o;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(o) : "r"(a), "r"(v) : "memory");
  return o;
}
__device__ __forceinline__ void st_remote64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// Sum over the block, to every thread; ends with a barrier, as block_inclusive_scan does.
__device__ __forceinline__ u64 block_sum(u64 v, u64 *scratch) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 t = 0;
  for (int w = 0; w < kSaWarps; ++w) t += scratch[w];
  __syncthreads();
  return t;
}

template <class T>
struct Row {
  static constexpr int N = Vec16<T>::N;
  const T *base;      // 16-byte aligned address at or below the row's first logit
  int sh, V;          // logits of the first vector that lie before the row
  int c0, c1;         // this CTA's vectors
  int v0, v1;         // this warp's, where the order of ids counts

  __device__ __forceinline__ Row(const T *row, int V_, int rank, int nc) : V(V_) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row);
    sh = static_cast<int>((a & 15u) / sizeof(T));
    base = row - sh;
    const int nvec = (V + sh + N - 1) / N;
    const int per = (nvec + nc - 1) / nc;
    c0 = min(rank * per, nvec);
    c1 = min(c0 + per, nvec);
    const int pw = (c1 - c0 + kSaWarps - 1) / kSaWarps;
    const int w = threadIdx.x >> 5;
    v0 = min(c0 + w * pw, c1);
    v1 = min(v0 + pw, c1);
  }
  static constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;   // -infinity
  // Vector j of the row.
  __device__ __forceinline__ uint4 vector(int j) const {
    return j * N - sh >= 0 && (j + 1) * N - sh <= V
               ? *reinterpret_cast<const uint4 *>(base + static_cast<int64_t>(j) * N)
               : edge(base + static_cast<int64_t>(j) * N, j * N - sh, V);
  }
  static __device__ __noinline__ uint4 edge(const T *p, int id, int V) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = kNone;
      if (sizeof(T) == 2) {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
        const uint32_t lo = id + 2 * i >= 0 && id + 2 * i < V ? h[2 * i] : 0xff80u;
        const uint32_t hi = id + 2 * i + 1 >= 0 && id + 2 * i + 1 < V ? h[2 * i + 1] : 0xff80u;
        w[i] = lo | hi << 16;
      } else if (id + i >= 0 && id + i < V) {
        w[i] = reinterpret_cast<const uint32_t *>(p)[i];
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ bool reaches(const uint4 &v, float low) {   // one of its logits is at or above `low`
    float x[N];
    Vec16<T>::unpack(v, x);
    bool any = false;
#pragma unroll
    for (int i = 0; i < N; ++i) any |= x[i] >= low;
    return any;
  }
  // f(x, id) for the logits of vector j, in order; a loop, so that f's code stands there once or twice.
  template <class F> __device__ __forceinline__ void elements(uint4 v, int j, F &&f) const {
    int id = j * N - sh;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 2) {
        f(__uint_as_float(v.x << 16), id);
        f(__uint_as_float(v.x & 0xffff0000u), id + 1);
        id += 2;
      } else {
        f(__uint_as_float(v.x), id++);
      }
      v.x = v.y;
      v.y = v.z;
      v.z = v.w;
    }
  }
  // f(x) for the logits of a vector, two in line.
  template <class F> static __device__ __forceinline__ void pairs(uint4 v, F &&f) {
#pragma unroll 1
    for (int i = 0; i < (sizeof(T) == 2 ? 4 : 2); ++i) {
      if (sizeof(T) == 2) {
        f(__uint_as_float(v.x << 16));
        f(__uint_as_float(v.x & 0xffff0000u));
        v.x = v.y;
        v.y = v.z;
        v.z = v.w;
      } else {
        f(__uint_as_float(v.x));
        f(__uint_as_float(v.y));
        v.x = v.z;
        v.y = v.w;
      }
    }
  }
  // Vector j; -infinity outside the CTA's range.
  __device__ __forceinline__ uint4 get_any(int j) const {
    return j < c1 ? vector(j) : make_uint4(kNone, kNone, kNone, kNone);
  }
  // Step g of 32 vectors from a0 on is a warp's whenever g is `me` modulo `of`; f(vector, j, i) for its i-th one, DEPTH of them
  // on their way: loads go straight to the registers they are used from (a copy from one to another would wait for them).
  // Steps that do not lie inside the row and before a1 (at most three) come after the others.
  template <int DEPTH, class F>
  __device__ __forceinline__ void steps(int a0, int a1, int me, int of, F &&f) const {
    const int lane = threadIdx.x & 31;
    const int first = a0 == 0 && sh != 0 ? 1 : 0;                     // step 0 holds the row's first, partial vector
    const int full = max(first, (min(a1, (V + sh) / N) - a0) / 32);   // steps [first, full) lie inside
    const int i0 = me < first ? 1 : 0, i1 = full > me ? (full - me + of - 1) / of : 0;
    const T *p = base + (static_cast<int64_t>(a0) + me * 32 + lane) * N;
    if (i1 > i0) {
      uint4 r[DEPTH];
      auto fetch = [&](int i) {
        return *reinterpret_cast<const uint4 *>(p + static_cast<int64_t>(min(i, i1 - 1)) * (of * 32 * N));
      };
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) r[k] = fetch(i0 + k);
#pragma unroll 1
      for (int i = i0; i < i1; i += DEPTH) {
#pragma unroll
        for (int k = 0; k < DEPTH; ++k)
          if (i + k < i1) {
            const uint4 v = r[k];
            r[k] = fetch(i + k + DEPTH);
            f(v, a0 + ((i + k) * of + me) * 32 + lane, i + k);
          }
      }
    }
    const int all = (a1 - a0 + 31) / 32;
#pragma unroll 1
    for (int i = i0 ? 0 : max(i1, 0); i * of + me < all; i = i0 && i == 0 ? max(i1, 1) : i + 1) {
      const int j = a0 + (i * of + me) * 32 + lane;
      f(j < a1 ? vector(j) : make_uint4(kNone, kNone, kNone, kNone), j, i);
    }
  }
  // The warps take a CTA's steps in turn, so that they read on side by side.
  template <int DEPTH, class F> __device__ __forceinline__ void stream(F &&f) const {
    steps<DEPTH>(c0, c1, threadIdx.x >> 5, kSaWarps, f);
  }
  // Each warp its own range, in the order of ids.
  template <int DEPTH, class F> __device__ __forceinline__ void in_order(F &&f) const { steps<DEPTH>(v0, v1, 0, 1, f); }
  // above(x) for the logits of a vector above `least`, and the number of those at it. Of 16-bit logits packed compares give
  // a mask first, and only its bits are looked at.
  template <class A> static __device__ __forceinline__ uint32_t kept(const uint4 &v, float least, A &&above) {
    if (sizeof(T) == 2) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      const __nv_bfloat162 l2 = __float2bfloat162_rn(least);
      // `least` is a logit or one of these limits, rounded up: a logit above it is above its rounding or equal to it
      const bool exact = __bfloat162float(__low2bfloat16(l2)) == least;
      uint32_t m = 0, e = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
        const uint32_t g = __hgt2_mask(x, l2), q = __heq2_mask(x, l2);
        m |= ((g & 1u) | ((g >> 15) & 2u)) << (2 * i);
        e |= ((q & 1u) | ((q >> 15) & 2u)) << (2 * i);
      }
      if (!exact) {
        if (__bfloat162float(__low2bfloat16(l2)) > least) m |= e;
        e = 0;
      }
      const uint32_t ties = __popc(e);
      while (m) {
        const int b = __ffs(m) - 1;
        m &= m - 1;
        const uint32_t lo = b & 2 ? v.y : v.x, hi = b & 2 ? v.w : v.z, word = b & 4 ? hi : lo;
        above(__uint_as_float(b & 1 ? word & 0xffff0000u : word << 16));
      }
      return ties;
    } else {
      uint32_t ties = 0;
      uint4 u = v;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const float x = __uint_as_float(u.x);
        u.x = u.y;
        u.y = u.z;
        u.z = u.w;
        if (x > least) above(x);
        else if (x == least) ++ties;
      }
      return ties;
    }
  }
  // g(x, id) for this lane's logits; ids outside the row come with -infinity.
  template <class G> __device__ __forceinline__ void each(G &&g) const {
    stream<2>([&](const uint4 &v, int j, int) {
      if (j < c1) elements(v, j, g);
    });
  }
  // g(x) in light passes.
  template <class G> __device__ __forceinline__ void each_light(G &&g) const {
    stream<4>([&](const uint4 &v, int, int) {
      float x[N];
      Vec16<T>::unpack(v, x);
#pragma unroll
      for (int i = 0; i < N; ++i) g(x[i]);
    });
  }
};

// x * f for a fraction f in [0, 1): rounded down, or up.
__device__ __forceinline__ u64 part_of(u64 x, float f, bool up) {
  if (!(f > 0.0f)) return 0;
  const uint32_t b = __float_as_uint(f);
  const int e = static_cast<int>(b >> 23);
  const uint32_t man = e ? ((b & 0x7fffffu) | 0x800000u) : (b & 0x7fffffu);
  const int sh = 150 - (e ? e : 1);
  const unsigned __int128 p = static_cast<unsigned __int128>(x) * man;
  if (sh >= 127) return up ? 1 : 0;
  const u64 q = static_cast<u64>(p >> sh);
  return q + ((up && (static_cast<unsigned __int128>(q) << sh) != p) ? 1 : 0);
}

template <class T>
struct Sampler {
  const Row<T> &row;
  Shared &s;
  int rank, nc, slot = 0;
  Weigh weigh;
  uint32_t *total;   // the cluster's histogram

  // Sums over the cluster, to every thread.
  __device__ u64 cluster_sum(u64 v) {
    const u64 b = block_sum(v, s.scan);
    if (nc == 1) return b;
    if (threadIdx.x == 0) s.sums[0][slot] = b;
    cluster_sync();
    u64 t = 0;
    for (int r = 0; r < nc; ++r) t += ld_remote64(remote(&s.sums[0][slot], r));
    slot ^= 1;
    return t;
  }
  __device__ uint32_t cluster_max(uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) s.scan[threadIdx.x >> 5] = v;
    __syncthreads();
    for (int w = 0; w < kSaWarps; ++w) v = max(v, static_cast<uint32_t>(s.scan[w]));
    __syncthreads();
    if (nc == 1) return v;
    if (threadIdx.x == 0) s.sums[0][slot] = v;
    cluster_sync();
    for (int r = 0; r < nc; ++r) v = max(v, static_cast<uint32_t>(ld_remote64(remote(&s.sums[0][slot], r))));
    slot ^= 1;
    return v;
  }
  // The cluster's histogram: s.hist of every CTA added up for every CTA.
  __device__ void join_hist(int bins = kBins) {
    __syncthreads();
    if (nc == 1) return;
    cluster_sync();
    const int per = (bins + nc - 1) / nc;
    for (int i = threadIdx.x; i < per; i += kSaThreads) {
      const int b = rank * per + i;
      if (b < bins) {
        uint32_t t = 0;
        for (int r = 0; r < nc; ++r) t += ld_remote32(remote(&s.hist[b], r));
        for (int r = 0; r < nc; ++r) st_remote32(remote(&s.joined[b], r), t);
      }
    }
    cluster_sync();
  }
  // The first bin at which the running sum (from `before`) of value(bin) reaches `target`, or kBins.
  template <class F> __device__ int first_bin(u64 before, u64 target, F &&value) {
    u64 v[kBinsPerThread], t = 0;
#pragma unroll
    for (int i = 0; i < kBinsPerThread; ++i) {
      v[i] = value(threadIdx.x * kBinsPerThread + i);
      t += v[i];
    }
    u64 run = before + block_inclusive_scan(t, s.scan) - t;
    if (threadIdx.x == 0) s.pick[0] = kBins;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBinsPerThread; ++i) {
      if (run < target && run + v[i] >= target) s.pick[0] = threadIdx.x * kBinsPerThread + i;
      run += v[i];
    }
    __syncthreads();
    const int b = static_cast<int>(s.pick[0]);
    __syncthreads();
    return b;
  }

  // Histogram of the distances to the maximum, 1/16 octave of weight a bin, of the logits from `least` on: their number,
  // and their weight (of those at `least`, only `ties` count where they are fewer). `total` holds the bins.
  struct Mass {
    u64 count, weight;
  };
  __device__ Mass histogram(float least, bool weights) {
    for (int i = threadIdx.x; i < kBins; i += kSaThreads) s.hist[i] = 0;
    __syncthreads();
    const float m = weigh.m, c = weigh.ch * kBinsPerOctave;
    u64 n = 0, w = 0;
    auto count = [&](float x) {
      ++n;
      const float y = (m - x) * c;
      atomicAdd(&s.hist[y < kBins - 1 ? static_cast<int>(y) : kBins - 1], 1u);
    };
    if (weights) {
      row.each([&](float x, int) {
        if (x >= least) {
          count(x);
          w += weigh(x);
        }
      });
    } else {
      row.each_light([&](float x) {
        if (x >= least) count(x);
      });
    }
    Mass r;
    r.count = cluster_sum(n);
    r.weight = weights ? cluster_sum(w) : 0;
    join_hist();
    return r;
  }
  // A logit at or above (up) or at or below all of the logits b bins from the maximum: rounding of the bin's number, of
  // the distance and of the sum widen it.
  __device__ float bin_edge(float b, bool up) const {
    const float d = fmaxf(b + (up ? -0.05f : 0.05f), 0.0f) / (weigh.ch * kBinsPerOctave);
    if (!(d < 1e38f)) return up ? weigh.m : -INFINITY;
    const float slack = (fabsf(weigh.m) + d) * 9.5e-7f;
    return up ? fminf(weigh.m, weigh.m - d + slack) : weigh.m - d - slack;
  }

  // Bounds of a bin's weight: that of one logit at its edge b / 16 octaves down, at most and at least (a logit's bin may be
  // off by 2^-19 of its distance, so 2^-12 of its weight).
  __device__ __forceinline__ u64 edge(int b) const {
    const int e = (b >> 4) + weigh.down;
    return e < 64 ? weigh.tab->q[(b & 15) * 4] >> e : u64(0);
  }
  __device__ __forceinline__ u64 bin_most(int b) const {
    const u64 w = edge(b);
    return total[b] * (w + (w >> 12) + 4);
  }
  __device__ __forceinline__ u64 bin_least(int b) const {
    const u64 w = edge(b + 1);
    return b == kBins - 1 || w < 8 ? u64(0) : total[b] * (w - (w >> 12) - 4);
  }
  // The bins in which the running weight can reach a target between `lo` and `hi`, and the interval of keys they can hold.
  __device__ void border_bins(u64 lo, u64 hi, int &b0, int &b1) {
    b0 = first_bin(0, lo, [&](int b) { return bin_most(b); });
    b1 = first_bin(0, hi, [&](int b) { return bin_least(b); });
  }
  __device__ void keys_of(int b0, int b1, uint32_t floor, uint32_t top, uint32_t &khi, uint32_t &klo) const {
    khi = top;
    klo = floor;
    if (b0 > 0) khi = min(top, order_key(bin_edge(static_cast<float>(b0), true)));
    if (b1 < kBins - 1) klo = max(floor, order_key(bin_edge(static_cast<float>(b1 + 1), false)));
    khi = max(khi, klo);
  }

  // After histogram(key_value(floor)): the least logit of the shortest run of the rank order, among logits whose key is
  // `floor` or more, that holds `target` tokens (by_weight false) or that much weight. Out: its key, how many tokens at it
  // and above it there are, and the weight above (by_weight). The run has to exist.
  __device__ void find(bool by_weight, u64 target, uint32_t floor, uint32_t top, uint32_t &key, u64 &at, u64 &above,
                       u64 &above_w) {
    int b0, b1;
    if (by_weight) {
      border_bins(target, target, b0, b1);
    } else {
      b0 = b1 = first_bin(0, target, [&](int b) { return static_cast<u64>(total[b]); });
    }
    uint32_t khi, klo;
    keys_of(b0, b1, floor, top, khi, klo);
    float known = INFINITY;   // what lies above it is in `above` and `above_w` already: khi only falls
    above = above_w = 0;
    while (true) {
      const uint32_t range = khi - klo;
      const int sh = max(0, 32 - __clz(range) - 11);
      const float vhi = key_value(khi), vlo = key_value(klo);
      for (int i = threadIdx.x; i < kBins; i += kSaThreads) s.hist[i] = 0;
      __syncthreads();
      u64 n = 0, w = 0;
      auto place = [&](float x) {
        if (x >= vlo) atomicAdd(&s.hist[(khi - order_key(x)) >> sh], 1u);
      };
      if (by_weight) {
        row.each([&](float x, int) {
          if (x > vhi) {
            if (x <= known) {
              ++n;
              w += weigh(x);
            }
          } else {
            place(x);
          }
        });
      } else {
        row.each_light([&](float x) {
          if (x > vhi) n += x <= known ? 1 : 0;
          else place(x);
        });
      }
      above += cluster_sum(n);
      if (by_weight) above_w += cluster_sum(w);
      known = vhi;
      join_hist();
      auto hi_key = [&](int b) { return khi - (static_cast<uint32_t>(b) << sh); };
      auto lo_key = [&](int b) {   // the last bin may reach past klo
        const u64 d = ((static_cast<u64>(b) + 1) << sh) - 1;
        return d > range ? klo : khi - static_cast<uint32_t>(d);
      };
      auto weight_at = [&](uint32_t k) { return weigh(key_value(k)); };
      auto used = [&](int b) { return total[b] != 0 && (static_cast<u64>(b) << sh) <= range; };
      if (by_weight) {
        const u64 more = sh == 0 ? 0 : 4;   // neighbours' weights may be out of order by their rounding
        b0 = first_bin(above_w, target, [&](int b) { return used(b) ? total[b] * (weight_at(hi_key(b)) + more) : u64(0); });
        b1 = sh == 0 ? b0 : first_bin(above_w, target, [&](int b) {
          const u64 lw = used(b) ? weight_at(lo_key(b)) : 0;
          return lw > more ? total[b] * (lw - more) : u64(0);
        });
      } else {
        b0 = b1 = first_bin(above, target, [&](int b) { return static_cast<u64>(total[b]); });
      }
      const int last = static_cast<int>(range >> sh);
      b0 = min(b0, last);
      b1 = min(b1, last);
      if (sh == 0) {
        u64 n_before = 0, w_before = 0;
        for (int b = threadIdx.x; b < b0; b += kSaThreads) {
          n_before += total[b];
          if (by_weight && total[b]) w_before += total[b] * weight_at(hi_key(b));
        }
        above += block_sum(n_before, s.scan);
        if (by_weight) above_w += block_sum(w_before, s.scan);
        key = hi_key(b0);
        at = total[b0];
        __syncthreads();
        return;
      }
      const uint32_t h = hi_key(b0), l = lo_key(b1);
      __syncthreads();
      if (h - l <= range / 2) {
        khi = h;
        klo = l;
        continue;
      }
      // the bounds leave more than half of the interval (weights far apart within a part): one halving by the exact sum
      const float mid = key_value(klo + range / 2);
      w = 0;
      row.each([&](float x, int) {
        if (x > mid) w += weigh(x);
      });
      if (cluster_sum(w) >= target) klo += range / 2 + 1;
      else khi = klo + range / 2;
    }
  }

  // One pass: this lane's largest logit, and the sum of 2^(x c - ref) with ref its running largest x c, rounded up, or -1e30 (ref
  // is a number of its own, so the exponents have one rounding; NaN where a logit is). Lane l keeps the maxima of the
  // warp's tiles l and l + 32: tile_iters iterations each.
  int tile_iters;
  float tile[2];
  __device__ void first_pass(float c, float &mx, float &ref, float &sum) {
    const int lane = threadIdx.x & 31;
    const int iters = ((row.c1 - row.c0 + 31) / 32 + kSaWarps - 1) / kSaWarps;
    tile_iters = max(1, (iters + kTiles - 1) / kTiles);
    mx = -INFINITY;
    ref = -1e30f;
    sum = 0.0f;
    tile[0] = tile[1] = -INFINITY;
    const F2 cc = f2(c, c);
    row.template stream<8>([&](const uint4 &raw, int, int q) {
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      float v, s0, s1;
      F2 t[4];
      if (sizeof(T) == 2) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(w);
        const __nv_bfloat162 top = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        const uint32_t u = *reinterpret_cast<const uint32_t *>(&top);
        v = fmaxf(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
      } else {
        v = fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])), fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
      }
      mx = fmaxf(mx, v);
      const float r = fmaxf(ref, __fmul_ru(v, c));   // upwards: no exponent is above 0
      const F2 nr = f2(-r, -r);
      constexpr int PAIRS = Row<T>::N / 2;
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        float a, b;
        split(fma2(sizeof(T) == 2 ? f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u))
                                  : f2(__uint_as_float(w[2 * i & 3]), __uint_as_float(w[(2 * i + 1) & 3])),
                   cc, nr), a, b);
        t[i] = f2(exp2_fast(a), exp2_fast(b));
      }
      F2 u = add2(t[0], t[1]);
      if (PAIRS == 4) u = add2(u, add2(t[2], t[3]));
      split(u, s0, s1);
      sum = fmaf(sum, exp2_fast(ref - r), s0 + s1);
      ref = r;
      const float top = warp_top(v);
      if (tile_iters > 1) q /= tile_iters;
      if (lane == (q & 31)) {
        if (q < 32) tile[0] = fmaxf(tile[0], top);
        else tile[1] = fmaxf(tile[1], top);
      }
    });
  }

  // The candidates in s.few.list in the rank order, in the CTA that has them: thread t gets the places 2 t and 2 t + 1 with
  // their weights (0 below `least`) and the running sums; its number of those from `least` on.
  __device__ int sort_list(int n, float least, u64 (&e)[2], u64 (&w)[2], u64 (&cum)[2]) {
    for (int i = threadIdx.x; i < n; i += kSaThreads) {
      const u64 v = s.few.list[i];
      int place = 0;
      for (int q = 0; q < n; ++q) place += s.few.list[q] > v ? 1 : 0;
      s.few.sorted[place] = v;
    }
    __syncthreads();
    int in = 0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = 2 * threadIdx.x + q;
      e[q] = i < n ? s.few.sorted[i] : 0;
      const float x = key_value(static_cast<uint32_t>(e[q] >> 32));
      const bool is = i < n && x >= least;
      w[q] = is ? weigh(x) : 0;
      in += is ? 1 : 0;
      s.few.w[i] = w[q];
    }
    cum[1] = block_inclusive_scan(w[0] + w[1], s.scan);
    cum[0] = cum[1] - w[1];
    return in;
  }
  __device__ __forceinline__ void push(float x, int id) {
    const u64 e = (static_cast<u64>(order_key(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
    const uint32_t at = nc > 1 ? add_remote32(remote(&s.few_count, 0), 1) : atomicAdd(&s.few_count, 1u);
    if (at < kFew) {
      if (nc > 1) st_remote64(remote(&s.few.list[at], 0), e);
      else s.few.list[at] = e;
    }
  }

  // The draw from few candidates: all logits at or above a bar that at least `n_bar` logits reach, gathered in the first CTA
  // and sorted there. It decides the row unless there are too many of them, or a border lies past them or within the error of
  // the row's approximate weight. True when the row is done. All of the cluster takes part.
  // The approximate weight of first_pass() in whole units, and what it is off by at most: 6 * 2^-24 of it for each of a lane's
  // vectors (a rounding, and where the reference changes an exponential's 2^-22 and a product's rounding), 64 * 2^-24 for
  // exponents off by 2^-20, joins, and weights cut to units.
  __device__ void about(float mass, u64 &sum, u64 &off) const {
    sum = static_cast<u64>(mass * static_cast<float>(u64(1) << (44 - weigh.down)));
    const u64 vectors = ((row.V / Row<T>::N + 1) / nc + 1) / kSaThreads + 2;
    off = (sum >> 24) * (6 * vectors + 64) + 1;
  }
  __device__ bool few(float mx, int n_bar, int k, bool greedy, float least, float tp, float u, float mass, float temp,
                      const SParams &p, int r) {
    const int lane = threadIdx.x & 31, t = threadIdx.x;
    // the bar: of the lanes' largest logits about the n_bar-th, by the upper 16 bits of its key
    const uint32_t mine = order_key(mx) >> 16;
    uint32_t bar = 0;
    if (t == 0) s.few_count = 0;
    const int share = (n_bar + nc - 1) / nc;   // every CTA brings its share
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t b = bar | (1u << bit);
      if (__syncthreads_count(mine >= b) >= share) bar = b;
    }
    if (nc > 1) {
      if (t == 0) s.sums[0][slot] = bar;
      cluster_sync();
      for (int c = 0; c < nc; ++c) bar = min(bar, static_cast<uint32_t>(ld_remote64(remote(&s.sums[0][slot], c))));
      slot ^= 1;
    }
    float low = bar > 0x00800000u >> 16 ? key_value(bar << 16) : -INFINITY;   // the keys below are -infinity's and NaN's
    if (row.V <= kFew) low = -3.402823466e38f;   // all of them
    else if (!(low > -1e30f)) return false;
    auto gather = [&](float x, int id) {
      if (x >= low) push(x, id);
    };
#pragma unroll 1
    for (int q0 = 0; q0 < kTiles; q0 += 32) {
      uint32_t mask = __ballot_sync(0xffffffffu, (q0 ? tile[1] : tile[0]) >= low);
      while (mask) {   // four tiles together
        int j[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          j[c] = mask ? row.c0 + ((q0 + __ffs(mask) - 1) * tile_iters * kSaWarps + (t >> 5)) * 32 + lane : row.c1;
          mask &= mask - 1;
        }
#pragma unroll 1
        for (int i = 0; i < tile_iters; ++i) {
          uint4 v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = row.get_any(j[c] + 32 * kSaWarps * i);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (Row<T>::reaches(v[c], low)) row.elements(v[c], j[c] + 32 * kSaWarps * i, gather);
        }
      }
    }
    if (nc > 1) cluster_sync();
    else __syncthreads();
    bool done = false;
    if (rank == 0) {
      const int n = s.few_count;
      if (n <= kFew) {
        u64 e[2], w[2], cum[2];
        const int in = sort_list(n, least, e, w, cum);
        if (t == 0) s.pick[2] = s.pick[3] = kFew;
        const int survive = static_cast<int>(block_sum(in, s.scan));   // a run from the first on
        const int most = k > 0 ? min(k, survive) : survive;
        // whether the candidates hold all that top_p is a share of
        const bool whole = k > 0 || least >= low;
        if ((most - 1) / 2 == t) s.pick[4] = (most - 1) & 1 ? cum[1] : cum[0];
        __syncthreads();
        u64 sum = s.pick[4], off = 0;
        if (!whole) about(mass, sum, off);
        int keep = most;
        // (the row's weight is not the survivors' where min_p drops some)
        bool sure = whole || (tp < 1.0f && least <= -3.402823466e38f && mass > 0.5f);
        if (tp < 1.0f) {
          const u64 lo = max(u64(1), part_of(sum - off, tp, true)), hi = max(u64(1), part_of(sum + off, tp, true));
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int i = 2 * t + q;
            if (i < most && cum[q] >= lo && cum[q] - w[q] < lo) s.pick[2] = i;
            if (i < most && cum[q] >= hi && cum[q] - w[q] < hi) s.pick[3] = i;
          }
          __syncthreads();
          sure = sure && s.pick[2] == s.pick[3] && s.pick[2] < kFew;
          keep = static_cast<int>(s.pick[2]) + 1;
        }
        if (greedy) {
          sure = true;
          keep = 1;
        }
        if (sure) {
          done = true;
          if ((keep - 1) / 2 == t) s.pick[5] = (keep - 1) & 1 ? cum[1] : cum[0];
          __syncthreads();
          const u64 kept = s.pick[5], target = part_of(kept, u, false);
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            const int i = 2 * t + q;
            if (i >= keep) break;
            const u64 eq = q ? e[1] : e[0], wq = q ? w[1] : w[0];
            const uint32_t inv = static_cast<uint32_t>(eq);
            u64 before = 0;   // kept weight of lower ids
            for (int o = 0; o < keep; ++o) before += static_cast<uint32_t>(s.few.sorted[o]) > inv ? s.few.w[o] : 0;
            if (greedy ? i == 0 : before <= target && target < before + wq) {
              p.tokens[r] = static_cast<int32_t>(0xffffffffu - inv);
              if (p.logprob)
                p.logprob[r] = greedy ? 0.0f : log_share(key_value(static_cast<uint32_t>(eq >> 32)), kept, temp);
              if (p.kept) p.kept[r] = keep;
            }
          }
        }
      }
      if (t == 0) s.few_done = done ? 1 : 0;
    }
    if (nc > 1) {
      cluster_sync();
      done = ld_remote32(remote(&s.few_done, 0)) != 0;
    }
    return done;
  }

  __device__ float log_share(float x, u64 kept, float temp) const {
    return static_cast<float>((static_cast<double>(x) - weigh.m) / temp -
                              log(ldexp(static_cast<double>(kept), weigh.down - 44)));
  }

  // What is kept: the logits above `least`, and of those at it (of weight w_least each) the first `ties` in id order.
  struct Kept {
    float least;
    u64 ties, w_least;
    // weight of `some` of the logits at `least`, `before` of which lie ahead
    __device__ __forceinline__ u64 of_ties(u64 before, u64 some) const {
      return before < ties ? min(some, ties - before) * w_least : 0;
    }
  };
  // Kept weight of this warp's range, what lies before it in the cluster, and all; logits at `least` in the range and
  // before it; the kept tokens' number.
  struct Sums {
    u64 mine, before, all, t_before, count;
  };
  template <bool ALL = false, class W> __device__ Sums sums(const Kept &kp, W &&weight) {
    u64 w = 0;
    uint32_t n = 0, e = 0;
    if (ALL) {   // nothing but -infinity is left out
      row.template in_order<2>([&](const uint4 &v, int, int) {
        row.pairs(v, [&](float x) {
          w += weigh.here(x);
          n += x > -INFINITY ? 1 : 0;
        });
      });
      return join_sums(kp, w, n, 0);
    }
    row.template in_order<2>([&](const uint4 &v, int, int) {
      e += Row<T>::kept(v, kp.least, [&](float x) {
        w += weight(x);
        ++n;
      });
    });
    return join_sums(kp, w, n, e);
  }
  // From each lane's weight and number of logits above `least` in its warp's range, and their number at it.
  __device__ Sums join_sums(const Kept &kp, u64 w, uint32_t n, uint32_t e) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    n = __reduce_add_sync(0xffffffffu, n);
    e = __reduce_add_sync(0xffffffffu, e);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    if (lane == 0) {
      s.scan[warp] = w;
      s.scan2[warp] = (static_cast<u64>(n) << 32) | e;
    }
    __syncthreads();
    u64 w_all = 0, c_all = 0, w_before = 0, c_before = 0;
    for (int i = 0; i < kSaWarps; ++i) {
      w_before += i < warp ? s.scan[i] : 0;
      c_before += i < warp ? s.scan2[i] : 0;
      w_all += s.scan[i];
      c_all += s.scan2[i];
    }
    __syncthreads();
    if (nc > 1) {
      if (threadIdx.x == 0) {
        s.sums[0][slot] = w_all;
        s.sums[2][slot] = c_all;
      }
      cluster_sync();
      w_all = c_all = 0;
      for (int c = 0; c < nc; ++c) {
        const u64 v = ld_remote64(remote(&s.sums[0][slot], c)), k = ld_remote64(remote(&s.sums[2][slot], c));
        w_before += c < rank ? v : 0;
        c_before += c < rank ? k : 0;
        w_all += v;
        c_all += k;
      }
      slot ^= 1;
    }
    constexpr u64 kLow = 0xffffffffu;
    Sums r;
    r.t_before = c_before & kLow;
    r.before = w_before + kp.of_ties(0, r.t_before);
    r.mine = w + kp.of_ties(r.t_before, e);
    r.all = w_all + kp.of_ties(0, c_all & kLow);
    r.count = (c_all >> 32) + min(c_all & kLow, kp.ties);
    return r;
  }
  // top_p's cut of the logits from `least` on and the sums of what is kept, in a histogram and two passes in the order of ids:
  // the first weighs every logit once and counts those in the interval of the border, which bounds of the row's weight
  // (first_pass()'s, or the bins') give ahead of it; the second gathers the part that the border is in, which is sorted.
  // False: too many logits there (equal ones, mostly).
  __device__ bool nucleus(float least, float tp, float mass, Kept &kp, Sums &sm) {
    const int t = threadIdx.x, warp = t >> 5;
    __syncthreads();   // few_count has been read
    if (t == 0) s.few_count = 0;
    histogram(least, false);
    u64 lo, hi;
    if (least <= -3.402823466e38f && mass > 0.5f) {
      u64 off;
      about(mass, lo, off);
      hi = lo + off;
      lo -= min(lo, off);
    } else {
      lo = hi = 0;
      for (int b = t; b < kBins; b += kSaThreads) {
        lo += bin_least(b);
        hi += bin_most(b);
      }
      lo = block_sum(lo, s.scan);
      hi = block_sum(hi, s.scan);
    }
    // from the top the bins' bounds are apart by 1/16 octave of the share, from the bottom by that of the rest: both
    int b0, b1;
    border_bins(max(u64(1), part_of(lo, tp, false)), max(u64(1), part_of(hi, tp, true)), b0, b1);
    const u64 rest_lo = lo - min(lo, part_of(lo, tp, true) + 1), rest_hi = hi - part_of(hi, tp, false);
    const int least_up = first_bin(0, rest_hi + 1, [&](int b) { return bin_least(kBins - 1 - b); });
    const int most_up = first_bin(0, rest_lo + 1, [&](int b) { return bin_most(kBins - 1 - b); });
    if (least_up < kBins) b0 = max(b0, kBins - 1 - least_up);
    if (most_up < kBins) b1 = min(b1, kBins - 1 - most_up);
    b0 = min(b0, kBins - 1);
    b1 = max(b0, b1);
    uint32_t khi, klo;
    keys_of(b0, b1, order_key(least), order_key(weigh.m), khi, klo);
    const uint32_t range = khi - klo;
    const int sh = max(0, 32 - __clz(range) - 11);
    const float vhi = key_value(khi), vlo = key_value(klo);
    __syncthreads();
    for (int i = t; i < kBins; i += kSaThreads) s.hist[i] = 0;
    __syncthreads();
    u64 all = 0, w = 0;
    uint32_t n = 0;
    row.template in_order<2>([&](const uint4 &v, int, int) {
      row.pairs(v, [&](float x) {
        const u64 one = x >= least ? weigh.here(x) : 0;
        all += one;
        if (x > vhi) {
          w += one;
          ++n;
        } else if (x >= vlo) {
          atomicAdd(&s.hist[(khi - order_key(x)) >> sh], 1u);
        }
      });
    });
    all = cluster_sum(all);
    const u64 first = cluster_sum(w), target = max(u64(1), part_of(all, tp, true));
    join_hist();
    if (first >= target) return false;
    auto hi_key = [&](int b) { return khi - (static_cast<uint32_t>(b) << sh); };
    auto lo_key = [&](int b) {
      const u64 d = ((static_cast<u64>(b) + 1) << sh) - 1;
      return d > range ? klo : khi - static_cast<uint32_t>(d);
    };
    auto used = [&](int b) { return total[b] != 0 && (static_cast<u64>(b) << sh) <= range; };
    const u64 more = sh == 0 ? 0 : 4;   // neighbours' weights may be out of order by their rounding
    b0 = first_bin(first, target, [&](int b) { return used(b) ? total[b] * (weigh(key_value(hi_key(b))) + more) : u64(0); });
    b1 = first_bin(first, target, [&](int b) {
      const u64 lw = used(b) ? weigh(key_value(lo_key(b))) : 0;
      return lw > more ? total[b] * (lw - more) : u64(0);
    });
    const int last = static_cast<int>(range >> sh);
    b1 = min(b1, last);
    u64 some = 0;
    for (int b = b0 + t; b <= b1; b += kSaThreads) some += total[b];
    if (b0 > last || block_sum(some, s.scan) > kFew) return false;
    const float ghi = key_value(hi_key(b0)), glo = key_value(lo_key(b1));
    row.template in_order<2>([&](const uint4 &v, int j, int) {
      row.elements(v, j, [&](float x, int id) {
        if (x <= vhi && x >= glo) {
          if (x > ghi) {
            w += weigh(x);
            ++n;
          } else {
            push(x, id);
          }
        }
      });
    });
    const u64 above = cluster_sum(w);
    if (t < kSaWarps) s.own_w[t] = s.own_n[t] = 0;
    if (t == 0) s.cut = 0;
    __syncthreads();
    if (rank == 0) {
      u64 e[2], we[2], cum[2];
      sort_list(min(s.few_count, static_cast<uint32_t>(kFew)), least, e, we, cum);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (above + cum[q] >= target && above + cum[q] - we[q] < target) s.cut = e[q];
    }
    if (nc > 1) cluster_sync();
    else __syncthreads();
    const u64 cut = ld_remote64(remote(&s.cut, 0));
    const uint32_t n_list = ld_remote32(remote(&s.few_count, 0));
    if (cut == 0 || n_list > kFew) return false;
    // the candidates above the border and at it, to the warps whose they are
    const int per = (row.c1 - row.c0 + kSaWarps - 1) / kSaWarps;
    u64 ties = 0;
    for (uint32_t i = t; i < n_list; i += kSaThreads) {
      const u64 e = ld_remote64(remote(&s.few.list[i], 0));
      const bool above_it = e >> 32 > cut >> 32, at_it = e >> 32 == cut >> 32;
      const int j = (static_cast<int>(0xffffffffu - static_cast<uint32_t>(e)) + row.sh) / Row<T>::N;
      if (j >= row.c0 && j < row.c1) {
        const int o = (j - row.c0) / per;
        if (above_it) atomicAdd(&s.own_w[o], weigh(key_value(static_cast<uint32_t>(e >> 32))));
        if (above_it || at_it) atomicAdd(&s.own_n[o], above_it ? u64(1) << 32 : u64(1));
      }
      ties += at_it && e >= cut ? 1 : 0;
    }
    kp.least = key_value(static_cast<uint32_t>(cut >> 32));
    kp.ties = block_sum(ties, s.scan);
    kp.w_least = weigh(kp.least);
    uint32_t at = 0;
    if ((t & 31) == 0) {
      w += s.own_w[warp];
      n += static_cast<uint32_t>(s.own_n[warp] >> 32);
      at = static_cast<uint32_t>(s.own_n[warp]);
    }
    sm = join_sums(kp, w, n, at);
    return true;
  }
  // The id at which the running kept weight in id order first passes `target`, and its logit; -1 if it never does. Every
  // thread of the cluster gets them.
  template <class W> __device__ int pick(const Sums &sm, const Kept &kp, u64 target, W &&weight, float &value) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sl = slot;
    slot ^= 1;
    __syncthreads();
    if (threadIdx.x == 0) {
      s.sums[1][sl] = ~u64(0);
      s.pick[0] = 0;
    }
    __syncthreads();
    if (lane == 0 && sm.before <= target && target < sm.before + sm.mine) {   // one warp of the cluster
      s.pick[0] = (static_cast<u64>(static_cast<uint32_t>(row.v0)) << 32) | static_cast<uint32_t>(row.v1);
      s.pick[1] = sm.before;
      s.pick[2] = sm.t_before;
    }
    __syncthreads();
    auto of_vector = [&](int j, int end, u64 &w, uint32_t &e) {   // a lane's vector: weight above `least`, logits at it
      if (j < end) e += Row<T>::kept(row.vector(j), kp.least, [&](float x) { w += weight(x); });
    };
    int a0 = static_cast<int>(s.pick[0] >> 32), a1 = static_cast<int>(s.pick[0] & 0xffffffffu);
    // its CTA: the warps share the range, then the part that the target lies in, until that is 32 vectors
    for (int step = 0; step < 10 && a1 - a0 > 32; ++step) {   // a sixteenth each time, of 32 vectors at least
      const u64 run0 = s.pick[1], ties0 = s.pick[2];
      const int per = ((a1 - a0 + kSaWarps - 1) / kSaWarps + 31) & ~31;
      const int w0 = min(a0 + warp * per, a1), w1 = min(w0 + per, a1);
      u64 w = 0;
      uint32_t e = 0;
#pragma unroll 1
      for (int j = w0 + lane; j < w1; j += 32) of_vector(j, w1, w, e);
      e = __reduce_add_sync(0xffffffffu, e);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      if (lane == 0) {
        s.scan[warp] = w;
        s.scan2[warp] = e;
      }
      __syncthreads();
      u64 run = run0, ties = ties0;
      for (int i = 0; i < warp; ++i) {
        run += s.scan[i] + kp.of_ties(ties, s.scan2[i]);
        ties += s.scan2[i];
      }
      __syncthreads();
      if (lane == 0 && run <= target && target < run + w + kp.of_ties(ties, e)) {   // one warp
        s.pick[0] = (static_cast<u64>(static_cast<uint32_t>(w0)) << 32) | static_cast<uint32_t>(w1);
        s.pick[1] = run;
        s.pick[2] = ties;
      }
      __syncthreads();
      a0 = static_cast<int>(s.pick[0] >> 32);
      a1 = static_cast<int>(s.pick[0] & 0xffffffffu);
    }
    if (a1 > a0 && warp == 0) {
      const u64 run = s.pick[1], ties = s.pick[2];
      u64 lw = 0;
      uint32_t le = 0;
      of_vector(a0 + lane, a1, lw, le);
      u64 wi = lw;
      uint32_t ei = le;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 v = shfl_up64(wi, o);
        const uint32_t c = __shfl_up_sync(0xffffffffu, ei, o);
        if (lane >= o) {
          wi += v;
          ei += c;
        }
      }
      // before this lane's vector
      u64 r = run + (wi - lw) + kp.of_ties(ties, ei - le), tb = ties + (ei - le);
      if (r <= target && target < r + lw + kp.of_ties(tb, le)) {   // one lane
        u64 hit = ~u64(0);
        row.elements(row.vector(a0 + lane), a0 + lane, [&](float x, int id) {
          if (x > kp.least) {
            r += weight(x);
          } else if (x == kp.least) {
            r += kp.of_ties(tb, 1);
            ++tb;
          }
          if (r > target && hit == ~u64(0))
            hit = (static_cast<u64>(static_cast<uint32_t>(id)) << 32) | __float_as_uint(x);
        });
        s.sums[1][sl] = hit;
      }
    }
    u64 got = ~u64(0);
    if (nc > 1) {
      cluster_sync();
      for (int r = 0; r < nc; ++r) got = min(got, ld_remote64(remote(&s.sums[1][sl], r)));
    } else {
      __syncthreads();
      got = s.sums[1][sl];
    }
    value = __uint_as_float(static_cast<uint32_t>(got));
    return got == ~u64(0) ? -1 : static_cast<int>(got >> 32);
  }

  // ---- 16-bit logits, counted by value: all sums from counts, each value weighed once
  static __device__ __forceinline__ int value_index(float x) {   // -1: another magnitude
    return bits_index(__float_as_uint(x) >> 16);
  }
  static __device__ __forceinline__ int bits_index(uint32_t u) {
    const uint32_t i = (u & 0x7fffu) - kFirstValue;
    return i >= kEndValue - kFirstValue ? -1 : static_cast<int>(i + (u >> 15) * kHalfValues);
  }
  static __device__ __forceinline__ float value_of(int b) {
    return __uint_as_float((b < kHalfValues ? kFirstValue + b : 0x8000u | (kFirstValue + (b - kHalfValues))) << 16);
  }
  // The k-th largest value's index.
  static __device__ __forceinline__ int ordered(int k) { return k < kHalfValues ? kHalfValues - 1 - k : k; }
  __device__ __forceinline__ u64 value_weight(float x) const {
    const int b = value_index(x);
    return b >= 0 ? s.weight[b] : weigh(x);
  }
  // Before the running sums of a thread's values; those between the signs, kept aside, count before the negative ones.
  static constexpr int kPer = kValues / kSaThreads;
  static_assert(kValues % kSaThreads == 0 && kHalfValues % kPer == 0, "a thread's values have one sign");
  struct Counted {
    u64 count, weight;             // before this thread's values
    u64 all_count, all_weight;
    u64 pos_count, pos_weight;     // of the positive values
    u64 odd_count, odd_weight;
  };
  // Counts the logits from `least` on. False: too many of other magnitudes, or some from 2^10 on (finite masks such as -1e9
  // among them: flat rows then take 3.2 ms for 2048 under top_p instead of 0.77 with a mask of -infinity).
  __device__ bool count_values(float least, Counted &c) {
    const int t = threadIdx.x;
    __syncthreads();
    for (int i = t; i < kValues; i += kSaThreads) s.hist[i] = 0;
    if (t == 0) s.odd_count = 0;
    __syncthreads();
    row.template stream<4>([&](const uint4 &v, int, int) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
        const int b = bits_index(u);
        if (b >= 0) atomicAdd(&s.hist[b], 1u);
        odd |= b < 0 && u != 0xff80u;   // -infinity counts nowhere
      }
      if (odd)
        row.elements(v, 0, [&](float x, int) {
          if (x >= least && value_index(x) < 0) {
            const uint32_t at = atomicAdd(&s.odd_count, 1u);
            if (at < kOdd) s.odd[at] = x;
          }
        });
    });
    __syncthreads();
    const uint32_t n = s.odd_count;
    // one word: the odd ones' number, and from 2^32 on whether this CTA cannot go on
    u64 word = t == 0 ? n + (n > kOdd ? u64(1) << 32 : 0) : 0, ow = 0;
    for (uint32_t i = t; i < min(n, static_cast<uint32_t>(kOdd)); i += kSaThreads) {
      const float x = s.odd[i];
      if (fabsf(x) >= 1024.0f) word += u64(1) << 32;
      ow += weigh(x);
    }
    c.odd_count = cluster_sum(word);
    if (c.odd_count >> 32) return false;
    c.odd_weight = c.odd_count ? cluster_sum(ow) : 0;
    join_hist(kValues);
    u64 cn = 0, cw = 0;
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
      const int b = ordered(t * kPer + i);
      const float x = value_of(b);
      const u64 k = x >= least ? total[b] : 0, w = k ? weigh(x) : 0;
      s.weight[b] = w;
      cn += k;
      cw += k * w;
    }
    c.count = block_inclusive_scan(cn, s.scan) - cn;
    c.weight = block_inclusive_scan(cw, s.scan) - cw;
    if (t * kPer == kHalfValues) {
      s.pick[2] = c.count;
      s.pick[3] = c.weight;
    }
    if (t == kSaThreads - 1) {
      s.pick[4] = c.count + cn;
      s.pick[5] = c.weight + cw;
    }
    __syncthreads();
    c.pos_count = s.pick[2];
    c.pos_weight = s.pick[3];
    c.all_count = s.pick[4] + c.odd_count;
    c.all_weight = s.pick[5] + c.odd_weight;
    if (t * kPer >= kHalfValues) {
      c.count += c.odd_count;
      c.weight += c.odd_weight;
    }
    __syncthreads();
    return true;
  }
  // find() over counted values. False: the border lies among those kept aside.
  __device__ bool find_value(const Counted &c, float least, bool by_weight, u64 target, uint32_t &key, u64 &at, u64 &above,
                             u64 &above_w) {
    u64 n = c.count, w = c.weight;
    if (threadIdx.x == 0) s.pick[0] = ~u64(0);
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
      const int b = ordered(threadIdx.x * kPer + i);
      const u64 k = value_of(b) >= least ? total[b] : 0, kw = k * s.weight[b];
      if (by_weight ? w < target && w + kw >= target : n < target && n + k >= target) {
        s.pick[0] = b;
        s.pick[1] = n;
        s.pick[2] = w;
      }
      n += k;
      w += kw;
    }
    __syncthreads();
    const u64 b = s.pick[0];
    above = s.pick[1];
    above_w = s.pick[2];
    const bool found = b < kValues;
    if (found) {
      key = order_key(value_of(static_cast<int>(b)));
      at = total[b];
    }
    __syncthreads();
    return found;
  }
};

// The draw from rows that few candidates do not decide. Out of line, so that the passes before it have their registers.
template <class T>
__device__ __noinline__ void draw_kept(const Row<T> row, Shared &s, int slot, const Weigh weigh, int k, float tp, float u,
                                       float least, float mass, float temp, const SParams &p, int r) {
  const int rank = cluster_rank(), nc = cluster_size();
  Sampler<T> a{row, s, rank, nc, slot, weigh, nc > 1 ? s.joined : s.hist, 0};
  const uint32_t best = order_key(weigh.m);
  float x_tok = 0.0f;
  int token = 0;
  u64 count = 0;
  // kept: the logits above `least`, and of those at it the first `ties` in id order
  constexpr u64 kAll = ~u64(0);
  u64 ties = kAll, total = 0;
  bool settled = false;
  const bool by_p = tp < 1.0f;
  const float least0 = least;
  // the steps on any way of counting: top_k's cut of `all` tokens, then top_p's
  auto cut_k = [&](uint32_t key, u64 at, u64 above) {
    least = key_value(key);
    ties = static_cast<u64>(k) - above < at ? static_cast<u64>(k) - above : kAll;
    count = k;
  };
  auto cut_p = [&](uint32_t key, u64 at, u64 above, u64 above_w, u64 target, u64 n_all) {
    const u64 each = a.weigh(key_value(key));
    const bool last = key_value(key) == least;   // the least logit that top_k left
    if (last) at = min(at, n_all - above);
    const u64 need = each ? min(at, (target - above_w + each - 1) / each) : at;
    count = above + need;
    ties = need < at || (last && ties != kAll) ? need : kAll;
    least = key_value(key);
  };
  typename Sampler<T>::Counted c;
  if (sizeof(T) == 2 && ((k > 0 && k < p.V) || by_p) && a.count_values(least, c)) {
    settled = true;
    uint32_t key;
    u64 at, above, above_w, weight = c.all_weight;
    count = c.all_count;
    if (k > 0 && static_cast<u64>(k) < count) {
      settled = a.find_value(c, least, false, k, key, at, above, above_w);
      if (settled) {
        cut_k(key, at, above);
        weight = above_w + (static_cast<u64>(k) - above) * a.weigh(least);
      }
    }
    if (settled && by_p) {
      const u64 target = max(u64(1), part_of(weight, tp, true)), n_all = count;
      settled = a.find_value(c, least0, true, target, key, at, above, above_w);
      if (settled) cut_p(key, at, above, above_w, target, n_all);
    }
    if (!settled) {
      least = least0;
      ties = kAll;
    }
  }
  const bool by_value = settled;
  typename Sampler<T>::Kept kp{};
  typename Sampler<T>::Sums sm{};
  const bool summed = sizeof(T) == 4 && by_p && !(k > 0 && k < p.V) && a.nucleus(least, tp, mass, kp, sm);
  if (!settled && !summed) {
    if (k > 0 && k < p.V) {
      count = a.histogram(least, false).count;
      if (static_cast<u64>(k) < count) {
        uint32_t key;
        u64 at, above, unused;
        a.find(false, k, order_key(least), best, key, at, above, unused);
        cut_k(key, at, above);
      }
    }
    if (by_p) {
      auto whole = a.histogram(least, true);
      u64 n_all = whole.count;
      if (ties != kAll) {   // tokens at the least logit that top_k does not keep
        whole.weight -= (whole.count - count) * a.weigh(least);
        n_all = count;
      }
      const u64 target = max(u64(1), part_of(whole.weight, tp, true));
      uint32_t key;
      u64 at, above, above_w;
      a.find(true, target, order_key(least), best, key, at, above, above_w);
      cut_p(key, at, above, above_w, target, n_all);
    }
  }
  if (!summed) kp = {least, ties, a.weigh(least)};
  auto draw = [&](auto &&weight) {
    count = sm.count;
    total = sm.all;
    token = a.pick(sm, kp, part_of(total, u, false), weight, x_tok);
  };
  auto counted = [&](float x) { return a.value_weight(x); };
  auto weighed = [&](float x) { return a.weigh(x); };
  if (by_value) {
    sm = a.sums(kp, counted);
    draw(counted);
  } else {
    if (!summed && kp.least <= -3.402823466e38f && ties == kAll) sm = a.template sums<true>(kp, weighed);
    else if (!summed) sm = a.sums(kp, weighed);
    draw(weighed);
  }
  if (rank == 0 && threadIdx.x == 0) {
    p.tokens[r] = max(token, 0);
    if (p.logprob) p.logprob[r] = a.log_share(x_tok, total, temp);
    if (p.kept) p.kept[r] = static_cast<int32_t>(count);
  }
}

template <class T>
__global__ void __launch_bounds__(kSaThreads, kSaCtas) sample_kernel(const __grid_constant__ SParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared &s = *reinterpret_cast<Shared *>(smem);
  grid_dependency_sync();
  const int nc = cluster_size(), rank = cluster_rank();
  const int r = blockIdx.x / nc;
  const Row<T> row(static_cast<const T *>(p.logits) + static_cast<int64_t>(r) * p.stride, p.V, rank, nc);
  const float temp = p.temp ? (p.temp[r] > 0.0f ? fmaxf(p.temp[r], 1e-36f) : 0.0f) : 1.0f;
  const int k = p.top_k ? p.top_k[r] : 0;
  const float tp = p.top_p ? p.top_p[r] : 1.0f, mp = p.min_p ? p.min_p[r] : 0.0f;
  const float ur = p.u[r], u = ur == ur ? fminf(ur, 0.99999994f) : 0.0f;
  Sampler<T> a{row, s, rank, nc, 0, {}, nc > 1 ? s.joined : s.hist, 0};
  const double cd = 1.4426950408889634 / static_cast<double>(temp > 0.0f ? temp : 1.0f);
  const float ch = static_cast<float>(cd);

  if (threadIdx.x < 64) {
    s.powers.f[threadIdx.x] = kPowers.f[threadIdx.x];
    s.powers.q[threadIdx.x] = kPowers.q[threadIdx.x];
  }
  // ---- the largest logit, whether the row is a distribution, and its weight to about 2^-17
  float mx, ref, mass;
  a.first_pass(fmaxf(ch, 1e-30f), mx, ref, mass);
  const int warp = threadIdx.x >> 5;
  float m = warp_top(mx);
  if ((threadIdx.x & 31) == 0) s.fscan[warp] = m;
  __syncthreads();
  for (int w = 0; w < kSaWarps; ++w) m = fmaxf(m, s.fscan[w]);
  if (nc > 1) {
    if (threadIdx.x == 0) s.sums[0][a.slot] = __float_as_uint(m);
    cluster_sync();
    for (int c = 0; c < nc; ++c) m = fmaxf(m, __uint_as_float(static_cast<uint32_t>(ld_remote64(remote(&s.sums[0][a.slot], c)))));
    a.slot ^= 1;
  }
  // (a row whose scaled maximum lies below -1e30 has no sum here; such rows do without)
  // nor does one that overflows when scaled: 1e30 marks it, and its NaNs are looked for below
  mass = warp_sum(!(ref < INFINITY) ? 1e30f : mass == 0.0f ? 0.0f : mass * exp2f(fmaf(-m, fmaxf(ch, 1e-30f), ref)));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.fscan[warp] = mass;
  __syncthreads();
  mass = 0.0f;
  for (int w = 0; w < kSaWarps; ++w) mass += s.fscan[w];
  if (nc > 1) {
    if (threadIdx.x == 0) s.sums[0][a.slot] = __float_as_uint(mass);
    cluster_sync();
    mass = 0.0f;
    for (int c = 0; c < nc; ++c) mass += __uint_as_float(static_cast<uint32_t>(ld_remote64(remote(&s.sums[0][a.slot], c))));
    a.slot ^= 1;
  }
  if (mass > 1e20f && m < INFINITY) {
    u64 nans = 0;
    row.each_light([&](float x) { nans += x != x ? 1 : 0; });
    mass = a.cluster_sum(nans) ? NAN : 0.0f;
  }
  const bool sound = mass == mass && fabsf(m) < INFINITY;
  // first_pass() took 1e-30 for smaller scales, at which logits of 1e28 and more below the largest still weigh as much
  if (sound && ch < 1e-30f) mass = 0.0f;
  float x_tok = m;
  int token = 0;
  float lp = 0.0f;
  u64 count = 0;
  bool done = false;
  // no weight reaches a min_p above 1: what is left is the first token, which is always kept
  const bool greedy = !(temp > 0.0f) || mp > 1.0f;
  float least = -3.402823466e38f;
  if (sound) {
    a.weigh = Weigh{m, ch, static_cast<float>(cd - static_cast<double>(ch)), 44 - p.qb, &s.powers};
    if (mp > 0.0f && !greedy) {
      if (threadIdx.x == 0)
        s.pick[1] = __float_as_uint(__double2float_ru(
            static_cast<double>(m) + static_cast<double>(temp) * log(static_cast<double>(mp))));
      __syncthreads();
      least = fminf(m, fmaxf(least, __uint_as_float(static_cast<uint32_t>(s.pick[1]))));
    }
    const bool by_k = k > 0 && k < p.V;
    if (greedy || p.V <= kFew || (by_k ? k <= kMaxFewK : (tp < 1.0f || mp > 0.0f)))
      done = a.few(mx, greedy ? 1 : by_k ? k : kFewBar, by_k ? k : 0, greedy, least, tp, u, mass, temp, p, r);
  }
  if (done) {
  } else if (!sound || greedy) {   // the first of the rank order
    // (in a row of -infinity and NaN the first -infinity, of NaN alone token 0)
    // padding is -infinity as well, but its ids come after those of the row's first one, or before 0: where the maximum is
    // -infinity, ids are looked at one by one
    if (m > -INFINITY) {
      const typename Sampler<T>::Kept kp{m, 1, 1};
      auto none = [](float) { return u64(0); };
      token = a.pick(a.sums(kp, none), kp, 0, none, x_tok);
    } else {
      int lowest = 0x7fffffff;
      row.each([&](float x, int id) {
        if (id >= 0 && id < p.V && x == -INFINITY) lowest = min(lowest, id);
      });
      lowest = static_cast<int>(0x7fffffffu - a.cluster_max(0x7fffffffu - static_cast<uint32_t>(lowest)));
      token = lowest < p.V ? lowest : 0;
    }
    lp = sound ? 0.0f : NAN;
    count = sound ? 1 : 0;
  } else {
    draw_kept<T>(row, s, a.slot, a.weigh, k, tp, u, least, mass, temp, p, r);
    done = true;
  }
  if (!done && rank == 0 && threadIdx.x == 0) {
    p.tokens[r] = max(token, 0);
    if (p.logprob) p.logprob[r] = lp;
    if (p.kept) p.kept[r] = static_cast<int32_t>(count);
  }
  if (nc > 1) cluster_sync();   // the others may still read this CTA's shared memory
}

constexpr int kSharedAll = sizeof(Shared) + kValues * sizeof(uint32_t);

template <class T> cudaError_t launch(const SParams &p, int nc, cudaStream_t s) {
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!attr_set[dev & 63]) {
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedAll);
    if (e != cudaSuccess) return e;
    attr_set[dev & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows * nc);
  cfg.blockDim = dim3(kSaThreads);
  cfg.dynamicSmemBytes = nc > 1 ? kSharedAll : sizeof(Shared);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nc;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
}

}  // namespace

cudaError_t launch_sample(const void *logits, int dtype, int V, int64_t stride, int rows, const float *u,
                          const float *temp, const int32_t *top_k, const float *top_p, const float *min_p,
                          int32_t *tokens, float *logprob, int32_t *kept, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  int bits = 0;
  while ((int64_t(1) << bits) < V) ++bits;
  const SParams p{logits, V, rows, std::min(44, 62 - bits), stride, u, temp, top_p, min_p, top_k, tokens, logprob, kept};
  // CTAs of a row: as many as fill the GPU once, but no slice below 2048 logits. More of them would spread flat rows among
  // others that end early (80 mixed fp32 rows: 4 CTAs 115 us where 3 took 131), but rows that few candidates decide then come in
  // two turns (51 us, 36).
  int nc = 1;
  nc = std::max(1, std::min({kMaxCluster, kSaCtas * device_sm_count() / rows, V / 2048}));
  if (nc > 8 && nc < kMaxCluster) nc = 8;   // past 8, a cluster of 16 or none
  return dtype == 0 ? launch<__nv_bfloat16>(p, nc, s) : launch<float>(p, nc, s);
}

}  // namespace kap
