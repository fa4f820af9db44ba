// k_packed.cu - 16-bit pages to packed 4-bit pages and back (sm_103a).
//
// A group is 64 dims of one token, head and tensor: lowest = min x, scale = the least bf16 that is not below
// (max - min) / 15, code = (x - lowest) / scale to nearest, ties to even. The scale rounds up, so the largest value has
// code 15 at most and every value is at most half a scale off. Everything is decided exactly: the two roundings of the
// scale are directed upwards (rounding up to fp32 and then to bf16 equals rounding up once, since every bf16 times 15 is
// an fp32), and a code is corrected by the sign of its exact remainder, so the packed page is a function of the values
// alone and equals what any exact arithmetic gives.
//
// Bound by HBM: a (page, head) of 128 dims reads 8192 and writes 2304 bytes. One warp takes one tensor of one (page,
// head): 8 lanes share a group (16 bytes of source and one word of codes each), so source loads are 512 contiguous
// bytes an instruction and all of them are in flight before the first is used.
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

// x - lowest, its code and the exact decision. h = scale / 2; all pre-multiplied by a power of two (exactly) for tiny
// and huge scales, so that the reciprocal and the difference stay finite.
__device__ __forceinline__ uint32_t code_of(float x, float lo, float k, float s, float inv, float h) {
  const float t = x * k - lo * k;
  float n = rintf(t * inv);
  const float rem = fmaf(-n, s, t);  // exact: n * s has 12 bits
  if (rem > h) n += 1.0f;
  else if (rem < -h) n -= 1.0f;
  else if (fabsf(rem) == h) {
    // on the border as far as t goes; t may have lost bits of x that lie below those of lowest (two-sum error)
    const float a = x * k, b = -lo * k, bb = t - a;
    const float e = (a - (t - bb)) + (b - bb);
    const float up = copysignf(1.0f, rem);  // the neighbour across the border
    if (e != 0.0f ? (e > 0.0f) == (rem > 0.0f) : (static_cast<int>(n) & 1) != 0) n += up;
  }
  return static_cast<uint32_t>(fminf(fmaxf(n, 0.0f), 15.0f));
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
    float x[8];
    Vec16<__nv_bfloat16>::unpack(v[j], x);
    float lo = x[0], hi = x[0], z = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo = fminf(lo, x[k]);
      hi = fmaxf(hi, x[k]);
      z = fmaf(x[k], 0.0f, z);  // NaN when any value is an infinity or a NaN
    }
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    lo += 0.0f;  // -0 stored as +0: which of the two a minimum returns is not defined
    // (max - min) / 15 in sixteenths, which no range overflows and which are exact for every bf16
    const float q = __fdiv_ru(__fadd_ru(hi * 0.0625f, -lo * 0.0625f), 0.9375f);
    // up to bf16: any low bits carry into the kept half
    uint32_t sb = (__float_as_uint(q) + 0xffffu) & 0xffff0000u;
    const bool bad = !(z == 0.0f);
    uint32_t word = 0;
    if (!bad && sb != 0) {
      const float s0 = __uint_as_float(sb);
      const float k = s0 < 0x1p-60f ? 0x1p64f : (s0 > 0x1p60f ? 0x1p-4f : 1.0f);
      const float s = s0 * k, inv = 1.0f / s, hf = 0.5f * s;
#pragma unroll
      for (int b = 0; b < 8; ++b) word |= code_of(x[b], lo, k, s, inv, hf) << (4 * b);
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
    const float s = param_scale(par[j]), lo = param_low(par[j]);
    float x[8];
#pragma unroll
    for (int b = 0; b < 8; ++b) x[b] = fmaf(s, static_cast<float>((word[j] >> (4 * b)) & 15u), lo);
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
