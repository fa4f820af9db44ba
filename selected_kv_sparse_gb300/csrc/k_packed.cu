// k_packed.cu - 16-bit pages to packed 4-bit pages and back (sm_103a).
//
// A group is 64 dims of one token, head and tensor: lowest = min x, scale = the least bf16 that is not below
// (max - min) / 15, code = (x - lowest) / scale to nearest, ties to even. The scale rounds up, so the largest value has
// code 15 at most and every value is at most half a scale off. Everything is decided exactly: the scale
// by comparing 15 times a bf16, which is an fp32, with the range rounded up, and the code by a correctly rounded quotient or
// by exact remainders, so the packed page is a function of the values alone and equals what exact arithmetic gives.
//
// Bound by HBM: a (page, head) of 128 dims reads 8192 and writes 2304 bytes. One warp takes one tensor of one (page,
// head): 8 lanes share a group (16 bytes of source and one word of codes each), so source loads are 512 contiguous
// bytes an instruction and all of them are in flight before the first is used.
// On a GB300, 2048 pages of 8 heads: packing 42 us (60% of the measured copy rate; 65 to 72% of the issue slots, since the
// scale, the reciprocal and the border test are worked out in all eight lanes of a group), reading back 28 us (90%); both
// after one another 66.7 us, 5.16 TB/s.
#include "kap_launch.h"
#include "kap_packed.cuh"

namespace kap {
namespace {

constexpr int kPackThreads = 256;

__device__ __forceinline__ bool pair_pages(const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int i,
                                           bool pack, int P16, int P4, int &p16, int &p4) {
  const int a = src[i], b = dst[i];
  p16 = pack ? a : b;
  p4 = (pack ? b : a) - P16;
  return p16 >= 0 && p16 < P16 && (pack ? b : a) >= P16 && p4 < P4;
}

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even

// The code of a value whose rounded quotient n left a remainder of at least half a scale (h): the neighbour where the
// remainder is larger, the even one where it is equal. t = x - lowest may have lost bits of x below lowest's last one:
// the two-sum error e then decides an equality.
__device__ __forceinline__ float settle(float n, float rem, float h, float t, float x, float lo) {
  const float r = fabsf(rem);
  if (r < h) return n;
  const float up = copysignf(1.0f, rem);
  if (r > h) return n + up;
  const float bb = t - x, e = (x - (t - bb)) + (-lo - bb);
  const bool over = e != 0.0f ? (e > 0.0f) == (rem > 0.0f) : (static_cast<int>(n) & 1) != 0;
  return over ? n + up : n;
}
// Settles a lane's eight values (a call of its own: rarely taken, and eight times in the caller).
__device__ __noinline__ uint32_t settle_word(uint32_t word, uint4 v, float k, float low, float s, float inv) {
  const float half = 0.5f * s;
#pragma unroll 1
  for (int b = 0; b < 8; ++b) {
    const uint32_t w = b < 4 ? (b < 2 ? v.x : v.y) : (b < 6 ? v.z : v.w);
    const float x = __uint_as_float((b & 1) ? w & 0xffff0000u : w << 16) * k, t = x - low;
    const float n = fmaf(t, inv, kMagic) - kMagic, rem = fmaf(-n, s, t);  // exact: n * s has 12 bits
    const float c = fminf(fmaxf(settle(n, rem, half, t, x, low), 0.0f), 15.0f);
    word = (word & ~(15u << (4 * b))) | (static_cast<uint32_t>(c) << (4 * b));
  }
  return word;
}

template <int D>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const __nv_bfloat16 *__restrict__ K,
                                                            const __nv_bfloat16 *__restrict__ V,
                                                            unsigned char *__restrict__ packed,
                                                            float *__restrict__ ksum, const int32_t *__restrict__ src,
                                                            const int32_t *__restrict__ dst, int n, int hkv, int P16,
                                                            int P4, int *err) {
  using L = PackedChunk<D>;
  constexpr int IT = kPage * D / 256;  // 16-byte source vectors of a lane
  grid_dependency_sync();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kPackThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<int64_t>(n) * hkv * 2) return;
  const int tensor = static_cast<int>(w & 1);
  const int64_t ph = w >> 1;
  const int i = static_cast<int>(ph / hkv), h = static_cast<int>(ph - static_cast<int64_t>(i) * hkv);
  int p16, p4;
  if (!pair_pages(src, dst, i, true, P16, P4, p16, p4)) {
    if (lane == 0) set_error(err, kErrPage);
    return;
  }
  const uint4 *from = reinterpret_cast<const uint4 *>((tensor ? V : K) +
                                                      (static_cast<size_t>(p16) * hkv + h) * (kPage * D));
  unsigned char *chunk = packed + (static_cast<size_t>(p4) * hkv + h) * L::BYTES;
  uint4 v[IT];
#pragma unroll
  for (int j = 0; j < IT; ++j) v[j] = __ldg(from + j * 32 + lane);
  if (tensor == 0 && ksum) {
    const float *a = ksum + (static_cast<size_t>(p16) * hkv + h) * D;
    float *b = ksum + (static_cast<size_t>(P16 + p4) * hkv + h) * D;
    for (int k = lane; k < D; k += 32) b[k] = a[k];
  }
#pragma unroll
  for (int j = 0; j < IT; ++j) {
    const int g = j * 4 + (lane >> 3);  // group: token g / NB, block g % NB
    const int tok = g / L::NB, blk = g - tok * L::NB;
    // extremes in bf16 pairs; NaN passes through, an infinity stays one
    const __nv_bfloat162 *h2 = reinterpret_cast<const __nv_bfloat162 *>(&v[j]);
    __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(h2[0], h2[1]), __hmin2_nan(h2[2], h2[3]));
    __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(h2[0], h2[1]), __hmax2_nan(h2[2], h2[3]));
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) {
      mn = __hmin2_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mx = __hmax2_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    const __nv_bfloat16 mn1 = __hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn));
    const __nv_bfloat16 mx1 = __hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx));
    const float lo = to_f(mn1) + 0.0f;  // -0 stored as +0: which of the two a minimum returns is not defined
    const float hi = to_f(mx1);
    const bool bad = !(fabsf(lo) < INFINITY) || !(fabsf(hi) < INFINITY);
    // the least bf16 b with 15 b >= max - min, both in sixteenths (exact for every bf16, and no range overflows): from
    // just below the quotient upwards; the difference is rounded up, which 15 b, an fp32, does not notice
    const float r16 = __fadd_ru(hi * 0.0625f, -lo * 0.0625f);
    uint32_t sb = __float_as_uint(r16 * 1.0666667f) & 0xffff0000u;
    if (__uint_as_float(sb) * 0.9375f < r16) sb += 0x10000u;
    if (__uint_as_float(sb) * 0.9375f < r16) sb += 0x10000u;
    uint32_t word = 0;
    if (!bad && sb != 0) {
      float x[8];
      Vec16<__nv_bfloat16>::unpack(v[j], x);
      float s = __uint_as_float(sb), low = lo, k = 1.0f;
      if (s < 0x1p-60f || s > 0x1p60f) {
        // tiny and huge scales: everything times a power of two (exactly), so that reciprocal and difference stay finite
        k = s < 1.0f ? 0x1p64f : 0x1p-4f;
        s *= k;
        low *= k;
#pragma unroll
        for (int b = 0; b < 8; ++b) x[b] *= k;
      }
      // the correctly rounded quotient t / s (one correction of t * (1 / s) by its exact remainder, Markstein's), then to
      // the nearest whole number: a border (k + 1/2) s gives k + 1/2 itself, so ties go to even
      float inv;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
      const F2 l2 = f2(-low, -low), inv2 = f2(inv, inv), mg = f2(kMagic, kMagic), ng = f2(-kMagic, -kMagic),
               s2 = f2(-s, -s);
      float n[8];
#pragma unroll
      for (int b = 0; b < 8; b += 2) {
        const F2 t2 = add2(f2(x[b], x[b + 1]), l2), q0 = mul2(t2, inv2), q1 = fma2(fma2(q0, s2, t2), inv2, q0);
        split(add2(add2(q1, mg), ng), n[b], n[b + 1]);
      }
      // four codes to a whole number below 2^16, in fp32, and its bits off the magic number
      const float a = fmaf(fmaf(fmaf(n[3], 16.0f, n[2]), 16.0f, n[1]), 16.0f, n[0]);
      const float c = fmaf(fmaf(fmaf(n[7], 16.0f, n[6]), 16.0f, n[5]), 16.0f, n[4]);
      word = __byte_perm(__float_as_uint(a + 8388608.0f), __float_as_uint(c + 8388608.0f), 0x5410);
      // A value below 2^-14 of the range may have lost bits in x - lowest, or lie nearer to a border than an fp32 quotient
      // tells (any other is at least 2^-22 of it away). All of these share one quotient, -lowest / scale, up to 2^-10:
      // only where that is within 2^-8 of a border are the lane's values settled by exact remainders.
      const float u0 = -low * inv;
      if (fabsf(u0 - rintf(u0)) > 0.5f - 0x1p-8f) {
        const __nv_bfloat162 ab =
            __hmin2(__hmin2(__habs2(h2[0]), __habs2(h2[1])), __hmin2(__habs2(h2[2]), __habs2(h2[3])));
        if (fminf(__low2float(ab), __high2float(ab)) < (hi - lo) * 0x1p-14f) word = settle_word(word, v[j], k, low, s, inv);
      }
    }
    *reinterpret_cast<uint32_t *>(chunk + (tensor ? L::OFF_V : 0) + blk * L::kBlock + tok * 32 + (lane & 7) * 4) = word;
    if ((lane & 7) == 0)
      *reinterpret_cast<uint32_t *>(chunk + (tensor ? L::OFF_VPAR : L::OFF_KPAR) + (blk * kPage + tok) * 4) =
          bad ? kNanParams : ((sb >> 16) | (__float_as_uint(lo) & 0xffff0000u));
  }
}

template <int D>
__global__ void __launch_bounds__(kPackThreads) unpack_kernel(__nv_bfloat16 *__restrict__ K,
                                                              __nv_bfloat16 *__restrict__ V,
                                                              const unsigned char *__restrict__ packed,
                                                              float *__restrict__ ksum,
                                                              const int32_t *__restrict__ src,
                                                              const int32_t *__restrict__ dst, int n, int hkv, int P16,
                                                              int P4, int *err) {
  using L = PackedChunk<D>;
  constexpr int IT = kPage * D / 256;
  grid_dependency_sync();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kPackThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<int64_t>(n) * hkv * 2) return;
  const int tensor = static_cast<int>(w & 1);
  const int64_t ph = w >> 1;
  const int i = static_cast<int>(ph / hkv), h = static_cast<int>(ph - static_cast<int64_t>(i) * hkv);
  int p16, p4;
  if (!pair_pages(src, dst, i, false, P16, P4, p16, p4)) {
    if (lane == 0) set_error(err, kErrPage);
    return;
  }
  const unsigned char *chunk = packed + (static_cast<size_t>(p4) * hkv + h) * L::BYTES;
  uint4 *to = reinterpret_cast<uint4 *>((tensor ? V : K) + (static_cast<size_t>(p16) * hkv + h) * (kPage * D));
  uint32_t word[IT], par[IT];
#pragma unroll
  for (int j = 0; j < IT; ++j) {
    const int g = j * 4 + (lane >> 3);
    const int tok = g / L::NB, blk = g - tok * L::NB;
    word[j] = __ldg(reinterpret_cast<const uint32_t *>(chunk + (tensor ? L::OFF_V : 0) + blk * L::kBlock + tok * 32 +
                                                       (lane & 7) * 4));
    par[j] = __ldg(reinterpret_cast<const uint32_t *>(chunk + (tensor ? L::OFF_VPAR : L::OFF_KPAR) +
                                                      (blk * kPage + tok) * 4));
  }
  if (tensor == 0 && ksum) {
    const float *a = ksum + (static_cast<size_t>(P16 + p4) * hkv + h) * D;
    float *b = ksum + (static_cast<size_t>(p16) * hkv + h) * D;
    for (int k = lane; k < D; k += 32) b[k] = a[k];
  }
#pragma unroll
  for (int j = 0; j < IT; ++j) {
    // a code in place k of a word, with the exponent of 2^23 over it, is 2^23 + 16^k code: off comes 2^23, and 16^-k goes
    // into the scale (exactly: the product and the sum are rounded once as for the bare code)
    const float s = param_scale(par[j]), lo = param_low(par[j]);
    const uint32_t w0 = word[j], w1 = w0 >> 16;
    const F2 l2 = f2(lo, lo), m2 = f2(-8388608.0f, -8388608.0f);
    const F2 sa = f2(s, s * 0x1p-4f), sb = f2(s * 0x1p-8f, s * 0x1p-12f);
    auto two = [&](uint32_t w, uint32_t ma, uint32_t mb, F2 sc, float &a, float &b) {
      const F2 c = add2(f2(__uint_as_float((w & ma) | 0x4b000000u), __uint_as_float((w & mb) | 0x4b000000u)), m2);
      split(fma2(c, sc, l2), a, b);
    };
    float x[8];
    if (s >= 0x1p-100f || !(s == s)) {
      two(w0, 0xfu, 0xf0u, sa, x[0], x[1]);
      two(w0, 0xf00u, 0xf000u, sb, x[2], x[3]);
      two(w1, 0xfu, 0xf0u, sa, x[4], x[5]);
      two(w1, 0xf00u, 0xf000u, sb, x[6], x[7]);
    } else {  // sixteenths of a scale this small would lose bits
#pragma unroll
      for (int b = 0; b < 8; ++b) x[b] = fmaf(s, static_cast<float>((w0 >> (4 * b)) & 15u), lo);
    }
    to[j * 32 + lane] = Vec16<__nv_bfloat16>::pack(x);
  }
}

}  // namespace

cudaError_t launch_pack(const PackedArgs &p, bool pack, const int32_t *src, const int32_t *dst, int n, int *err,
                        cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(n) * p.pool.hkv * 2;
  const int64_t blocks = (warps + kPackThreads / 32 - 1) / (kPackThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  __nv_bfloat16 *k = static_cast<__nv_bfloat16 *>(const_cast<void *>(p.pool.k));
  __nv_bfloat16 *v = static_cast<__nv_bfloat16 *>(const_cast<void *>(p.pool.v));
  unsigned char *c = static_cast<unsigned char *>(p.packed);
  const int hkv = p.pool.hkv, P16 = p.pool.num_pages, P4 = p.num_packed;
  if (pack && p.pool.d == 128)
    return launch_pdl(pack_kernel<128>, grid, dim3(kPackThreads), 0, s, k, v, c, p.pool.ksum, src, dst, n, hkv, P16, P4,
                      err);
  if (pack) return launch_pdl(pack_kernel<64>, grid, dim3(kPackThreads), 0, s, k, v, c, p.pool.ksum, src, dst, n, hkv, P16, P4, err);
  if (p.pool.d == 128)
    return launch_pdl(unpack_kernel<128>, grid, dim3(kPackThreads), 0, s, k, v, c, p.pool.ksum, src, dst, n, hkv, P16,
                      P4, err);
  return launch_pdl(unpack_kernel<64>, grid, dim3(kPackThreads), 0, s, k, v, c, p.pool.ksum, src, dst, n, hkv, P16, P4,
                    err);
}

}  // namespace kap
