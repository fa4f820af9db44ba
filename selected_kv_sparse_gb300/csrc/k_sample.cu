// k_sample.cu - sampling of tokens with temperature, top-k, min-p and top-p from given random numbers (sm_103a).
//
// Mathematics, for a row of logits x with the largest m at temperature T: w_i = exp((x_i - m) / T). The rank order is
// logit descending, lower id first. The tokens among the first top_k that weigh min_p or more are a run of that order from
// its start, and so is the shortest part of it that holds top_p of its weight: what is kept is a least logit, all tokens
// above it and the first few ids of those at it. The token drawn is the first in id order at which the running sum of the
// kept weights passes u times their sum.
// Weights are whole numbers, 2^-44 of the largest each (fewer bits past 2^18 tokens, so that sums stay below 2^62), so
// sums do not depend on their order and every border is decided as 64-bit floating point would decide it.
//
// The least logit is found from counts: a histogram of the distances to the maximum in 1/16 octaves of weight bounds the
// sums at its bins' edges, which leaves an interval of logits; that is cut by its bits, 2048 parts at a time, until a part
// is one logit.
// A row belongs to a cluster of CTAs, each with a slice of it; they add up their parts through one another's shared
// memory.
#include "kap_device.cuh"
#include "kap_launch.h"

#include <algorithm>

namespace kap {
namespace {

constexpr int kSaThreads = 512;
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

// exp((x - m) / T) as a whole number of 2^-qb, right to about 2^-40 of itself and a half unit, for x <= m that is no NaN:
// with y = (m - x) log2 e / T as a sum of two fp32, k the nearest whole number to 64 y and r = y - k / 64,
//   2^-y = 2^(-k/64) (1 - t + t^2/2 - t^3/6 + t^4/24),  t = r ln 2 <= 0.0055, t's leading term again as two fp32.
// From y = 22 on (weights below 2^-22, units 2^-44) the exponential unit's 2^-22 of the value is below a unit.
struct Weigh {
  float m, ch, cl;   // largest logit; log2 e / T
  int down;          // 44 - qb
  const Powers *tab;
  __device__ __forceinline__ u64 operator()(float x) const {
    // m - x, exactly (two-sum)
    const float dh = m - x, bb = m - dh, dl = (m - (dh + bb)) + (bb - x);
    const float yh = dh * ch;
    const float yl = fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch);
    if (!(yh < 62.0f)) return 0;   // also an infinite distance
    constexpr float kLn2h = 0.693147182464599609375f, kLn2l = -1.904654323148236017e-9f;
    u64 w;
    int e;
    if (yh >= 22.0f) {
      float v;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(44.0f - yh));   // the difference is exact
      v = fmaf(v, -yl * kLn2h, v);
      return (static_cast<u64>(__float_as_uint(v + 12582912.0f) - 0x4b400000u) + ((1u << down) >> 1)) >> down;
    }
    const float kf = fmaf(yh, 64.0f, 12582912.0f);   // 1.5 * 2^23: the sum's low bits are the nearest whole number
    const int k = static_cast<int>(__float_as_uint(kf) - 0x4b400000u);
    const float r = fmaf(kf - 12582912.0f, -0.015625f, yh);
    const float th = r * kLn2h, tl = fmaf(r, kLn2h, -th) + fmaf(r, kLn2l, yl * kLn2h);
    const float q = th * th * fmaf(th, fmaf(th, 0.0416666679f, -0.166666672f), 0.5f) - tl;
    const float2 f = tab->f[k & 63];
    const float ph = f.x * -th;
    const float pl = fmaf(f.x, -th, -ph) + fmaf(f.x, q, f.y * -th);
    // ph + pl in units of 2^-44, through the low bits of sums at 3 (unit 2^-22) and at 3 * 2^-22
    const float u = ph + pl, ub = u - ph, ul = (ph - (u - ub)) + (pl - ub);
    const float s1 = u + 3.0f;
    const int i1 = static_cast<int>(__float_as_uint(s1) - 0x40400000u);
    const float rest = (u - (s1 - 3.0f)) + ul;
    const int i2 = static_cast<int>(__float_as_uint(rest + 7.152557373046875e-7f) - 0x35400000u);
    w = tab->q[k & 63] + static_cast<u64>(static_cast<int64_t>(i1) * (1 << 22) + i2);
    e = (k >> 6) + down;
    return (w + ((u64(1) << e) >> 1)) >> e;
  }
};

struct Shared {
  uint32_t hist[kBins], total[kBins];
  u64 scan[kSaWarps];
  u64 sums[2][2];   // values for the other CTAs, in turn: a slot is written again two exchanges later
  u64 pick[6];
};

__device__ __forceinline__ u64 shfl_up64(u64 v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

// Sum over the block, to every thread.
__device__ __forceinline__ u64 block_sum(u64 v, u64 *scratch) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 t = 0;
  for (int w = 0; w < kSaWarps; ++w) t += scratch[w];
  return t;
}

template <class T>
struct Row {
  static constexpr int N = Vec16<T>::N;
  const T *base;      // 16-byte aligned address at or below the row's first logit
  int sh, V;          // logits of the first vector that lie before the row
  int v0, v1;         // this warp's vectors

  __device__ __forceinline__ Row(const T *row, int V_, int rank, int nc) : V(V_) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row);
    sh = static_cast<int>((a & 15u) / sizeof(T));
    base = row - sh;
    const int nvec = (V + sh + N - 1) / N;
    const int per = (nvec + nc - 1) / nc;
    const int c0 = min(rank * per, nvec), c1 = min(c0 + per, nvec);
    const int pw = (c1 - c0 + kSaWarps - 1) / kSaWarps;
    const int w = threadIdx.x >> 5;
    v0 = min(c0 + w * pw, c1);
    v1 = min(v0 + pw, c1);
  }
  // The N logits of vector j; -infinity outside the row.
  __device__ __forceinline__ void load(int j, float *x) const {
    const int id = j * N - sh;
    if (inside(j)) {
      Vec16<T>::unpack(at(j), x);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        x[i] = (id + i >= 0 && id + i < V) ? to_f(base[static_cast<int64_t>(j) * N + i]) : -INFINITY;
    }
  }
  // f(x, id) for this thread's logits, which are in its warp's range; ids outside the row come with -infinity. The next
  // vector is on its way while f sees this one.
  template <class F> __device__ __forceinline__ void each(F &&f) const {
    int j = v0 + (threadIdx.x & 31);
    uint4 raw{};
    if (j < v1 && inside(j)) raw = at(j);
#pragma unroll 1
    for (; j < v1; j += 32) {
      float x[N];
      if (inside(j)) Vec16<T>::unpack(raw, x);
      else load(j, x);
      if (j + 32 < v1 && inside(j + 32)) raw = at(j + 32);
#pragma unroll
      for (int i = 0; i < N; ++i) f(x[i], j * N - sh + i);
    }
  }
  // f(x) for the same logits in light passes: four vectors on their way together.
  template <class F> __device__ __forceinline__ void each_light(F &&f) const {
#pragma unroll 1
    for (int j = v0 + (threadIdx.x & 31); j < v1; j += 128) {
      uint4 raw[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + 32 * k < v1 && inside(j + 32 * k)) raw[k] = at(j + 32 * k);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (j + 32 * k >= v1) break;
        float x[N];
        if (inside(j + 32 * k)) Vec16<T>::unpack(raw[k], x);
        else load(j + 32 * k, x);
#pragma unroll
        for (int i = 0; i < N; ++i) f(x[i]);
      }
    }
  }
  __device__ __forceinline__ bool inside(int j) const { return j * N - sh >= 0 && (j + 1) * N - sh <= V; }
  __device__ __forceinline__ uint4 at(int j) const {
    return *reinterpret_cast<const uint4 *>(base + static_cast<int64_t>(j) * N);
  }
};

template <class T>
struct Sampler {
  const Row<T> &row;
  Shared &s;
  int rank, nc, slot = 0;
  Weigh weigh;

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
  // The cluster's histogram: s.hist of every CTA added up into s.total of every CTA.
  __device__ void join_hist() {
    __syncthreads();
    if (nc == 1) {
      for (int i = threadIdx.x; i < kBins; i += kSaThreads) s.total[i] = s.hist[i];
      __syncthreads();
      return;
    }
    cluster_sync();
    const int per = (kBins + nc - 1) / nc;
    for (int i = threadIdx.x; i < per; i += kSaThreads) {
      const int b = rank * per + i;
      if (b < kBins) {
        uint32_t t = 0;
        for (int r = 0; r < nc; ++r) t += ld_remote32(remote(&s.hist[b], r));
        for (int r = 0; r < nc; ++r) st_remote32(remote(&s.total[b], r), t);
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
  // and their weight (of those at `least`, only `ties` count where they are fewer). s.total holds the bins.
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

  // After histogram(key_value(floor)): the least logit of the shortest run of the rank order, among logits whose key is
  // `floor` or more, that holds `target` tokens (by_weight false) or that much weight. Out: its key, how many tokens at it
  // and above it there are, and the weight above (by_weight). The run has to exist.
  __device__ void find(bool by_weight, u64 target, uint32_t floor, uint32_t top, uint32_t &key, u64 &at, u64 &above,
                       u64 &above_w) {
    int b0, b1;
    if (by_weight) {
      // the weight at a bin's edge, b / 16 octaves down; a logit's bin may be off by 2^-19 of its distance (2^-12 of a weight)
      auto edge = [&](int b) {
        const int e = (b >> 4) + weigh.down;
        return e < 64 ? weigh.tab->q[(b & 15) * 4] >> e : u64(0);
      };
      b0 = first_bin(0, target, [&](int b) {
        const u64 w = edge(b);
        return s.total[b] * (w + (w >> 12) + 4);
      });
      b1 = first_bin(0, target, [&](int b) {
        const u64 w = edge(b + 1);
        return b == kBins - 1 || w < 8 ? u64(0) : s.total[b] * (w - (w >> 12) - 4);
      });
    } else {
      b0 = b1 = first_bin(0, target, [&](int b) { return static_cast<u64>(s.total[b]); });
    }
    // the interval of keys that the bins b0 .. b1 can hold
    uint32_t khi = top, klo = floor;
    if (b0 > 0) khi = min(top, order_key(bin_edge(static_cast<float>(b0), true)));
    if (b1 < kBins - 1) klo = max(floor, order_key(bin_edge(static_cast<float>(b1 + 1), false)));
    khi = max(khi, klo);
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
            ++n;
            w += weigh(x);
          } else {
            place(x);
          }
        });
      } else {
        row.each_light([&](float x) {
          if (x > vhi) ++n;
          else place(x);
        });
      }
      above = cluster_sum(n);
      above_w = by_weight ? cluster_sum(w) : 0;
      join_hist();
      auto hi_key = [&](int b) { return khi - (static_cast<uint32_t>(b) << sh); };
      auto lo_key = [&](int b) {   // the last bin may reach past klo
        const u64 d = ((static_cast<u64>(b) + 1) << sh) - 1;
        return d > range ? klo : khi - static_cast<uint32_t>(d);
      };
      auto weight_of = [&](uint32_t k) { return weigh(key_value(k)); };
      auto used = [&](int b) { return s.total[b] != 0 && (static_cast<u64>(b) << sh) <= range; };
      if (by_weight) {
        const u64 more = sh == 0 ? 0 : 4;   // neighbours' weights may be out of order by their rounding
        b0 = first_bin(above_w, target, [&](int b) { return used(b) ? s.total[b] * (weight_of(hi_key(b)) + more) : u64(0); });
        b1 = sh == 0 ? b0 : first_bin(above_w, target, [&](int b) {
          const u64 lw = used(b) ? weight_of(lo_key(b)) : 0;
          return lw > more ? s.total[b] * (lw - more) : u64(0);
        });
      } else {
        b0 = b1 = first_bin(above, target, [&](int b) { return static_cast<u64>(s.total[b]); });
      }
      const int last = static_cast<int>(range >> sh);
      b0 = min(b0, last);
      b1 = min(b1, last);
      if (sh == 0) {
        u64 n_before = 0, w_before = 0;
        for (int b = threadIdx.x; b < b0; b += kSaThreads) {
          n_before += s.total[b];
          if (by_weight && s.total[b]) w_before += s.total[b] * weight_of(hi_key(b));
        }
        above += block_sum(n_before, s.scan);
        if (by_weight) above_w += block_sum(w_before, s.scan);
        key = hi_key(b0);
        at = s.total[b0];
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

  // The id at which the running sum in id order of amount(x, id) first passes `target`, and that logit; -1 if it never
  // does. Every thread of the cluster gets them.
  template <class F> __device__ int locate(u64 target, F &&amount, float &value) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    u64 w = 0;
    row.each([&](float x, int id) { w += amount(x, id); });
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    __syncthreads();
    if (lane == 0) s.scan[warp] = w;
    __syncthreads();
    u64 mine = 0, all = 0;
    for (int i = 0; i < kSaWarps; ++i) {
      mine += i < warp ? s.scan[i] : 0;
      all += s.scan[i];
    }
    const int sl = slot;
    slot ^= 1;
    if (threadIdx.x == 0) {
      s.sums[0][sl] = all;
      s.sums[1][sl] = ~u64(0);
    }
    if (nc > 1) {
      cluster_sync();
      for (int r = 0; r < rank; ++r) mine += ld_remote64(remote(&s.sums[0][sl], r));
    } else {
      __syncthreads();
    }
    if (mine <= target && target < mine + w) {   // one warp of the cluster
      u64 run = mine;
      for (int j0 = row.v0; j0 < row.v1; j0 += 32) {
        const int j = j0 + lane;
        float x[Row<T>::N];
        u64 a = 0;
        if (j < row.v1) {
          row.load(j, x);
#pragma unroll
          for (int i = 0; i < Row<T>::N; ++i) a += amount(x[i], j * Row<T>::N - row.sh + i);
        }
        u64 incl = a;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 v = shfl_up64(incl, o);
          if (lane >= o) incl += v;
        }
        if (run + incl - a <= target && target < run + incl) {   // one lane
          u64 r = run + incl - a;
          u64 hit = ~u64(0);
#pragma unroll
          for (int i = 0; i < Row<T>::N; ++i) {
            const int id = j * Row<T>::N - row.sh + i;
            r += amount(x[i], id);
            if (r > target && hit == ~u64(0))
              hit = (static_cast<u64>(static_cast<uint32_t>(id)) << 32) | __float_as_uint(x[i]);
          }
          s.sums[1][sl] = hit;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
        if (run > target) break;
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
__global__ void __launch_bounds__(kSaThreads, 2) sample_kernel(const SParams p) {
  __shared__ Shared s;
  grid_dependency_sync();
  const int nc = cluster_size(), rank = cluster_rank();
  const int r = blockIdx.x / nc;
  const Row<T> row(static_cast<const T *>(p.logits) + static_cast<int64_t>(r) * p.stride, p.V, rank, nc);
  const float temp = p.temp ? (p.temp[r] > 0.0f ? fmaxf(p.temp[r], 1e-36f) : 0.0f) : 1.0f;
  const int k = p.top_k ? p.top_k[r] : 0;
  const float tp = p.top_p ? p.top_p[r] : 1.0f, mp = p.min_p ? p.min_p[r] : 0.0f;
  Sampler<T> a{row, s, rank, nc, 0, {}};

  // ---- the largest logit, and whether the row is a distribution
  float mx = -INFINITY;
  bool nan = false;
  row.each_light([&](float x) {
    nan |= x != x;
    mx = fmaxf(mx, x);
  });
  uint32_t best = order_key(mx);
  best = __reduce_max_sync(0xffffffffu, best);
  nan = __any_sync(0xffffffffu, nan);
  if ((threadIdx.x & 31) == 0) s.scan[threadIdx.x >> 5] = (static_cast<u64>(best) << 1) | (nan ? 1 : 0);
  __syncthreads();
  best = 0;
  for (int w = 0; w < kSaWarps; ++w) {
    best = max(best, static_cast<uint32_t>(s.scan[w] >> 1));
    nan |= (s.scan[w] & 1) != 0;
  }
  if (nc > 1) {
    if (threadIdx.x == 0) s.sums[0][a.slot] = (static_cast<u64>(best) << 1) | (nan ? 1 : 0);
    cluster_sync();
    for (int c = 0; c < nc; ++c) {
      const u64 v = ld_remote64(remote(&s.sums[0][a.slot], c));
      best = max(best, static_cast<uint32_t>(v >> 1));
      nan |= (v & 1) != 0;
    }
    a.slot ^= 1;
  }
  const float m = key_value(best);
  const bool sound = !nan && fabsf(m) < INFINITY;
  float x_tok = m;
  int token;
  float lp = 0.0f;
  u64 count = 0;
  if (!sound || !(temp > 0.0f)) {   // the first of the rank order
    // (in a row of -infinity and NaN the first -infinity, of NaN alone token 0)
    token = a.locate(0, [&](float x, int id) -> u64 { return id >= 0 && id < p.V && x == m ? 1 : 0; }, x_tok);
    lp = sound ? 0.0f : NAN;
    count = sound ? 1 : 0;
  } else {
    const double cd = 1.4426950408889634 / static_cast<double>(temp);
    const float ch = static_cast<float>(cd);
    a.weigh = Weigh{m, ch, static_cast<float>(cd - static_cast<double>(ch)), 44 - p.qb, &kPowers};
    float least = -3.402823466e38f;
    if (mp > 0.0f) {
      if (threadIdx.x == 0)
        s.pick[1] = __float_as_uint(__double2float_ru(
            static_cast<double>(m) + static_cast<double>(temp) * log(fmin(static_cast<double>(mp), 1.0))));
      __syncthreads();
      least = fminf(m, fmaxf(least, __uint_as_float(static_cast<uint32_t>(s.pick[1]))));
    }
    // kept: the logits above `least`, and of those at it the first `ties` in id order
    uint32_t floor = order_key(least);
    constexpr u64 kAll = ~u64(0);
    u64 ties = kAll, total = 0;
    int id_cut = 0x7fffffff;
    bool counted = false, summed = false;
    const bool by_p = tp < 1.0f;
    if (k > 0 && k < p.V) {
      const auto mass = a.histogram(least, false);
      count = mass.count;
      counted = true;
      if (static_cast<u64>(k) < count) {
        uint32_t key;
        u64 at, above, unused;
        a.find(false, k, floor, best, key, at, above, unused);
        floor = key;
        least = key_value(key);
        ties = static_cast<u64>(k) - above < at ? static_cast<u64>(k) - above : kAll;
        count = k;
      }
    }
    if (by_p) {
      auto mass = a.histogram(least, true);
      const u64 w_least = a.weigh(least);
      u64 n_all = mass.count;
      if (ties != kAll) {   // tokens at the least logit that top_k does not keep
        const u64 dropped = mass.count - count;
        mass.weight -= dropped * w_least;
        n_all = count;
      }
      const u64 target = max(u64(1), part_of(mass.weight, tp, true));
      uint32_t key;
      u64 at, above, above_w;
      a.find(true, target, floor, best, key, at, above, above_w);
      const u64 each = a.weigh(key_value(key));
      if (key == floor) at = min(at, n_all - above);
      const u64 need = each ? min(at, (target - above_w + each - 1) / each) : at;
      count = above + need;
      total = above_w + need * each;
      counted = summed = true;
      ties = need < at || (key == floor && ties != kAll) ? need : kAll;
      floor = key;
      least = key_value(key);
    }
    if (ties != kAll) {
      float unused;
      id_cut = a.locate(ties - 1, [&](float x, int) -> u64 { return x == least ? 1 : 0; }, unused);
    }
    auto weight = [&](float x, int id) -> u64 {
      return x > least || (x == least && id <= id_cut) ? a.weigh(x) : u64(0);
    };
    if (!counted) {   // the kept tokens' number and weight come with the sums of the draw below
      u64 n = 0;
      row.each_light([&](float x) { n += x >= least ? 1 : 0; });
      count = a.cluster_sum(n);
    }
    if (!summed) {
      u64 w = 0;
      row.each([&](float x, int id) { w += weight(x, id); });
      total = a.cluster_sum(w);
    }
    const float u = p.u[r];
    token = a.locate(part_of(total, u == u ? fminf(u, 0.99999994f) : 0.0f, false), weight, x_tok);
    if (rank == 0 && threadIdx.x == 0)
      lp = static_cast<float>((static_cast<double>(x_tok) - m) / temp - log(ldexp(static_cast<double>(total), -p.qb)));
  }
  if (rank == 0 && threadIdx.x == 0) {
    p.tokens[r] = max(token, 0);
    if (p.logprob) p.logprob[r] = lp;
    if (p.kept) p.kept[r] = static_cast<int32_t>(count);
  }
  if (nc > 1) cluster_sync();   // the others may still read this CTA's shared memory
}

template <class T> cudaError_t launch(const SParams &p, int nc, cudaStream_t s) {
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!attr_set[dev & 63]) {
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set[dev & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows * nc);
  cfg.blockDim = dim3(kSaThreads);
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
  // CTAs of a row: as many as fill the GPU twice, but no slice below 2048 logits
  int nc = 1;
  while (nc < kMaxCluster && rows * nc * 2 <= 2 * device_sm_count() && V / (nc * 2) >= 2048) nc *= 2;
  return dtype == 0 ? launch<__nv_bfloat16>(p, nc, s) : launch<float>(p, nc, s);
}

}  // namespace kap
