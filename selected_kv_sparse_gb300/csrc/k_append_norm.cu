// k_append_norm.cu - KV append with per-head norms of queries and keys and rotary positions on several axes (sm_103a).
//
// Mathematics, for a row x of one head: r = (mean x^2 + eps)^-1/2, y_i = x_i r w_i (y = x where no weight is given), then
// the pairs (y_i, y_{i + d/2}) turn by pos[axis(i)] * inv_freq[i]; one rounding into the pool's type at the end.
// The angle is formed in turns and in 64-bit whole numbers: F_i = inv_freq[i] / 2 pi, of which only the fraction matters
// beside a whole position, is held to 2^-64 turns, and pos * F_i modulo 2^64 is the angle's fraction of a turn without
// a rounding: at any position it is off by no more than position * 2^-63 turns (for frequencies up to 1). An fp32 product would be off by 2^-24
// of the angle, 1/128 at position 131072. Its top 32 bits go to sincospif.
//
// Bound by HBM: every row is read and written once. A lane holds 8 pairs (16 bytes on either side of a bf16 row), so a row
// is d / 16 lanes and its sum of squares three or two shuffles. Sines and cosines are formed once a token, by all
// threads into shared memory, while the first rows are in flight. 16384 tokens of 32 + 16 bf16 rows of 128 take 79 us (75% of
// the measured copy rate; 82 with 4 tokens a CTA, 77 with two rows a lane on their way, but then calls of few tokens take 3
// to 6% more); 4 tokens 2.9 us, a launch and two dependent loads. Frequencies turned into fractions in fp64: 2 to 12% more.
#include "kap_device.cuh"
#include "kap_launch.h"

namespace kap {
namespace {

constexpr int kAnThreads = 256;
constexpr int kAnWarps = kAnThreads / 32;
constexpr int kMaxTok = 8;  // tokens of a CTA: a warp a token

// 8 consecutive elements
template <class T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float *o) const { Vec16<__nv_bfloat16>::unpack(w, o); }
  __device__ __forceinline__ void set(const float *v) { w = Vec16<__nv_bfloat16>::pack(v); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = w; }
};
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void get(float *o) const {
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
  }
  __device__ __forceinline__ void set(const float *v) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void store(float *p) const {
    *reinterpret_cast<float4 *>(p) = a;
    *reinterpret_cast<float4 *>(p + 4) = b;
  }
};

// The fraction of a turn that a position adds at frequency f (radians a position), times 2^64 and rounded down: f's 24 bits
// times 2^66 / 2 pi, which is right to 2^-64 of itself. In whole numbers, since fp64 is slow here. A frequency that is not
// finite gives 0.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint32_t u = __float_as_uint(f), e = (u >> 23) & 0xffu;
  if (e == 0xffu) return 0;
  const uint64_t m = e ? (u & 0x7fffffu) | 0x800000u : u & 0x7fffffu;   // |f| = m 2^(max(e, 1) - 150)
  constexpr uint64_t kTurn = 0xa2f9836e4e44152aull;
  const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
  const int sh = 152 - static_cast<int>(max(e, 1u));                    // of the 88 bits, to the right
  uint64_t t;
  if (sh >= 128) t = 0;
  else if (sh >= 64) t = hi >> (sh - 64);
  else if (sh > 0) t = (lo >> sh) | (hi << (64 - sh));
  else t = sh > -64 ? lo << -sh : 0;
  return u >> 31 ? 0 - t : t;
}

// CTA (x, y): tokens [x * tt, x * tt + tt), of each the row groups y, y + gridDim.y, ... A group is the rows that a warp
// takes in one step. Rows of a token: hq queries, hkv keys, hkv values.
template <class T, int D>
__global__ void __launch_bounds__(kAnThreads) append_norm_kernel(const NormAppendArgs a, T *__restrict__ Kp,
                                                                 T *__restrict__ Vp, int num_pages, int hkv, int hq,
                                                                 int tt, int *err) {
  constexpr int HALF = D / 2;
  constexpr int LPR = HALF / 8;      // lanes of a row
  constexpr int RPW = 32 / LPR;      // rows of a warp's step
  __shared__ uint64_t s_turn[HALF];
  __shared__ int s_axis[HALF];
  __shared__ float2 s_cs[kMaxTok][HALF];  // cosine, sine
  __shared__ __align__(16) float s_w[2][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_sync();
  const int t0 = blockIdx.x * tt;
  const int ntok = min(tt, a.num_tokens - t0);
  const int wpt = kAnWarps / tt;     // warps of a token
  const int t = warp / wpt;          // this warp's token
  const bool live = t < ntok;
  const int rows = hq + 2 * hkv;
  const int step = wpt * gridDim.y * RPW;
  const int sub = lane & (LPR - 1);
  int row = ((warp - t * wpt) * gridDim.y + blockIdx.y) * RPW + lane / LPR;
  const int64_t tok = t0 + t;
  int64_t slot = -1;
  if (live) {
    slot = a.slots[tok * a.tok_stride];
    if (slot >= static_cast<int64_t>(num_pages) * kPage) {
      if (lane == 0) set_error(err, kErrPage);
      slot = -1;
    }
  }
  auto source = [&](int r) -> const T * {
    const T *p;
    if (r < hq) p = static_cast<const T *>(a.q) + tok * a.q_stride + static_cast<int64_t>(r) * D;
    else if (r < hq + hkv) p = static_cast<const T *>(a.k) + tok * a.k_stride + static_cast<int64_t>(r - hq) * D;
    else p = static_cast<const T *>(a.v) + tok * a.v_stride + static_cast<int64_t>(r - hq - hkv) * D;
    return p + sub * 8;
  };
  auto wanted = [&](int r) { return live && r < rows && (r < hq || slot >= 0); };
  Eight<T> x0, x1;
  if (wanted(row)) {
    const T *p = source(row);
    x0.load(p);
    x1.load(p + HALF);
  }
  for (int i = tid; i < HALF; i += kAnThreads) {
    s_turn[i] = turn_fraction(a.inv_freq[i]);
    const int ax = a.freq_axis ? a.freq_axis[i] : 0;
    s_axis[i] = (ax >= 0 && ax < a.num_axes) ? ax : -1;
  }
  for (int i = tid; i < 2 * D; i += kAnThreads) {
    const float *w = i < D ? a.q_weight : a.k_weight;
    s_w[i / D][i % D] = w ? w[i % D] : 1.0f;
  }
  __syncthreads();
  for (int i = tid; i < ntok * HALF; i += kAnThreads) {
    const int u = i / HALF, f = i - u * HALF;
    const int ax = s_axis[f];
    float cs = 1.0f, sn = 0.0f;
    if (ax >= 0) {
      const int p = a.pos[ax * a.axis_stride + (t0 + u) * static_cast<int64_t>(a.tok_stride)];
      const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(p)) * s_turn[f];
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
    }
    s_cs[u][f] = make_float2(cs, sn);
  }
  __syncthreads();
  if (!live) return;
  float2 cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = s_cs[t][sub * 8 + i];
  const int64_t page = slot >= 0 ? slot / kPage : 0;
  const int off = static_cast<int>(slot - page * kPage);
  // every lane of the warp takes the same number of steps: a row's lanes join in its sum by shuffles
  for (int base = row - lane / LPR; base < rows; base += step, row += step) {
    const bool mine = wanted(row);
    const Eight<T> y0 = x0, y1 = x1;
    if (wanted(row + step)) {   // the next row's loads
      const T *p = source(row + step);
      x0.load(p);
      x1.load(p + HALF);
    }
    T *dst = nullptr;
    if (mine) {
      if (row < hq) {
        dst = static_cast<T *>(a.q_out) + tok * a.q_out_stride + static_cast<int64_t>(row) * D;
      } else {
        const int h = row < hq + hkv ? row - hq : row - hq - hkv;
        dst = (row < hq + hkv ? Kp : Vp) + ((page * hkv + h) * kPage + off) * D;
      }
      dst += sub * 8;
    }
    const bool turned = row < hq + hkv;
    float u[8], v[8];
    if (mine) {
      y0.get(u);
      y1.get(v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = v[i] = 0.0f;
    }
    const int which = row < hq ? 0 : 1;
    if (a.q_weight || a.k_weight) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(u[i], u[i], fmaf(v[i], v[i], s));
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (turned && (which == 0 ? a.q_weight : a.k_weight)) {
        const float r = rsqrtf(fmaf(s, 1.0f / D, a.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[i] = u[i] * r * s_w[which][sub * 8 + i];
          v[i] = v[i] * r * s_w[which][HALF + sub * 8 + i];
        }
      }
    }
    if (mine) {
      Eight<T> o0, o1;
      if (turned) {
        float x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) rope_rotate(u[i], v[i], cs[i].x, cs[i].y, x[i], y[i]);
        o0.set(x);
        o1.set(y);
      } else {   // values are copied unchanged
        o0 = y0;
        o1 = y1;
      }
      o0.store(dst);
      o1.store(dst + HALF);
    }
  }
}

}  // namespace

cudaError_t launch_append_norm(const PoolArgs &p, const NormAppendArgs &a, int *err, cudaStream_t s) {
  if (a.num_tokens <= 0) return cudaSuccess;
  const int hq = a.q ? p.hq : 0;
  const int rows = hq + 2 * p.hkv;
  const int rpw = 32 / (p.d / 16);
  const int groups = (rows + rpw - 1) / rpw;       // warp steps of a token
  const int sms = device_sm_count();
  // few tokens: a CTA a token, its rows shared out over CTAs; many, or fewer steps a token than warps: up to 8 tokens a CTA
  // (1000 tokens of 12 fp32 rows of 64, two steps: a CTA a token 7.75 us, four tokens 3.35)
  int tt = 1;
  while (tt < kMaxTok && (a.num_tokens / (2 * tt) >= 4 * sms || kAnWarps / tt > groups)) tt *= 2;
  const int gx = (a.num_tokens + tt - 1) / tt;
  const int wpt = kAnWarps / tt;
  int gy = 1;
  while (gx * gy < 2 * sms && gy * wpt < groups) gy *= 2;
  const dim3 grid(gx, gy);
#define KAP_APPEND_NORM(TT, D)                                                                                    \
  launch_pdl(append_norm_kernel<TT, D>, grid, dim3(kAnThreads), 0, s, a, static_cast<TT *>(const_cast<void *>(p.k)), \
             static_cast<TT *>(const_cast<void *>(p.v)), p.num_pages, p.hkv, hq, tt, err)
  if (p.dtype == 0 && p.d == 128) KAP_APPEND_NORM(__nv_bfloat16, 128);
  else if (p.dtype == 0) KAP_APPEND_NORM(__nv_bfloat16, 64);
  else if (p.d == 128) KAP_APPEND_NORM(float, 128);
  else KAP_APPEND_NORM(float, 64);
#undef KAP_APPEND_NORM
  return cudaGetLastError();
}

}  // namespace kap
