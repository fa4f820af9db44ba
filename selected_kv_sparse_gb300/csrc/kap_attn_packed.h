// kap_attn_packed.h - what the two attention kernels over packed pages share (internal to the library).
#pragma once

#include <cuda_bf16.h>

#include "kap_launch.h"

namespace kap {

constexpr int kMaxCtas = 320;   // records of a launch beside one per row: CTAs of the widest grid
constexpr int kMaxRest = 8;     // slices of a row in the launch that takes what the other kernel leaves
constexpr float kNoMax = -1e30f;  // reference of a column that has seen nothing

struct AttnParams {
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
  int *counters;  // one per row
  float2 *ml;     // [slot][columns]: maximum (log2 units) and sum of a record
  float *part;    // [slot][columns][d]: its sums of values
  int ncol;       // columns of a record: G * max_q
  int by_row;     // a CTA a row, no shares
  // > 0: the windows' wholly visible packed pages are another kernel's; the others are taken in this many slices a row,
  // whose records lie in the slots from rest_slot + row * rest
  int rest;
  size_t rest_slot;
  int *err;
};

// Verification windows of 9 to 64 columns at head_dim 128 (k_attn_packed_tc.cu); p.rest records a row are merged in.
cudaError_t launch_attn_packed_tc(const AttnParams &p, cudaStream_t s);

}  // namespace kap
