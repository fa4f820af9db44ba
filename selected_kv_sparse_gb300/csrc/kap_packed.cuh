// kap_packed.cuh - the layout of a packed page, shared by the kernels that write and read it (sm_103a).
//
// The chunk of one (page, KV head) holds NB = d / 64 blocks of K codes [16 tokens][32 bytes], as many of V codes, then
// the K and the V parameters [NB][16 tokens], one word each: (scale, lowest value) in bf16, the scale in the low half.
// A code c stands for lowest + scale * c. The K and V of a (page, head) lie in one piece of 1152 * NB bytes, so one bulk
// copy brings them; a block is the unit that tensor-core fragments are taken from without bank conflicts.
#pragma once

#include "kap_device.cuh"

namespace kap {

template <int D>
struct PackedChunk {
  static constexpr int NB = D / 64;
  static constexpr int kBlock = kPage * 32;             // code bytes of one block
  static constexpr int OFF_V = NB * kBlock;
  static constexpr int OFF_KPAR = 2 * NB * kBlock;
  static constexpr int OFF_VPAR = OFF_KPAR + NB * kPage * 4;
  static constexpr int BYTES = OFF_VPAR + NB * kPage * 4;
};
static_assert(PackedChunk<64>::BYTES == 1152 && PackedChunk<128>::BYTES == 2304, "packed chunk layout");

constexpr uint32_t kNanParams = 0x7fff7fffu;  // (scale, lowest) of a group without finite values: reads back as NaN

__device__ __forceinline__ float param_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float param_low(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace kap
