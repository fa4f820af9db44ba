// k_logprobs.cu - log probabilities of given tokens, entropy, rank and the best alternatives (sm_103a).
//
// One CTA per row: the row's maximum, then sum exp(x - max), the entropy's sum and the token's rank in a second pass,
// then one pass per alternative for the next token in the order (logit descending, lower id first, NaN last).
#include "kap_device.cuh"
#include "kap_launch.h"

namespace kap {
namespace {

constexpr int kLpThreads = 256;

__device__ __forceinline__ unsigned long long rank_key(float x, int t) {
  return (static_cast<unsigned long long>(order_key(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(t));
}

template <class V, class F>
__device__ __forceinline__ V block_reduce(V v, F f, V *scratch) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = scratch[0];
  for (int w = 1; w < kLpThreads / 32; ++w) v = f(v, scratch[w]);
  __syncthreads();
  return v;
}

template <class T>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const T *__restrict__ logits, int V, int64_t stride,
                                                              const int32_t *__restrict__ tokens, int top_n,
                                                              float *__restrict__ lp, float *__restrict__ ent,
                                                              int32_t *__restrict__ rank,
                                                              int32_t *__restrict__ top_ids,
                                                              float *__restrict__ top_lp) {
  __shared__ unsigned long long s_u[kLpThreads / 32];
  __shared__ float s_f[kLpThreads / 32];
  grid_dependency_sync();
  const int row = blockIdx.x;
  const T *x = logits + row * stride;
  const int tok = tokens[row];
  const bool has = tok >= 0 && tok < V;
  const float xt = has ? to_f(x[tok]) : -INFINITY;
  const unsigned long long kt = has ? rank_key(xt, tok) : 0ull;
  float m = -INFINITY, bad = 0.0f;
  int before = 0;
  for (int t = threadIdx.x; t < V; t += kLpThreads) {
    const float v = to_f(x[t]);
    m = fmaxf(m, v);
    if (!(v < INFINITY)) bad = 1.0f;
    before += rank_key(v, t) > kt;
  }
  auto fmx = [](float a, float b) { return fmaxf(a, b); };
  auto add = [](float a, float b) { return a + b; };
  m = block_reduce(m, fmx, s_f);
  bad = block_reduce(bad, fmx, s_f);
  before = static_cast<int>(block_reduce<unsigned long long>(
      before, [](unsigned long long a, unsigned long long b) { return a + b; }, s_u));
  const bool none = bad != 0.0f || m == -INFINITY;
  float s = 0.0f, h = 0.0f;
  for (int t = threadIdx.x; t < V; t += kLpThreads) {
    const float d = to_f(x[t]) - m, e = expf(d);
    s += e;
    if (e > 0.0f) h = fmaf(e, d, h);
  }
  s = block_reduce(s, add, s_f);
  h = block_reduce(h, add, s_f);
  const float ls = logf(s);
  if (threadIdx.x == 0) {
    lp[row] = !has ? -INFINITY : none ? NAN : (xt - m) - ls;
    if (ent) ent[row] = none ? NAN : ls - h / s;
    if (rank) rank[row] = has ? before : V;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < top_n; ++k) {
    unsigned long long best = 0;
    for (int t = threadIdx.x; t < V; t += kLpThreads) {
      const unsigned long long key = rank_key(to_f(x[t]), t);
      if (key < last && key > best) best = key;
    }
    best = block_reduce(best, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; }, s_u);
    const int t = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
    if (threadIdx.x == 0) {
      top_ids[row * top_n + k] = t;
      top_lp[row * top_n + k] = none ? NAN : (to_f(x[t]) - m) - ls;
    }
    last = best;
  }
}

}  // namespace

size_t logprobs_workspace_bytes(int rows, int vocab) {
  (void)vocab;
  return static_cast<size_t>(rows) * 16;
}

cudaError_t launch_logprobs(const void *logits, int dtype, int V, int64_t stride, int rows, const int32_t *tokens,
                            int top_n, float *lp, float *ent, int32_t *rank, int32_t *top_ids, float *top_lp, void *ws,
                            cudaStream_t s) {
  (void)ws;
  if (dtype == 0)
    return launch_pdl(logprobs_kernel<__nv_bfloat16>, dim3(rows), dim3(kLpThreads), 0, s,
                      static_cast<const __nv_bfloat16 *>(logits), V, stride, tokens, top_n, lp, ent, rank, top_ids,
                      top_lp);
  return launch_pdl(logprobs_kernel<float>, dim3(rows), dim3(kLpThreads), 0, s, static_cast<const float *>(logits), V,
                    stride, tokens, top_n, lp, ent, rank, top_ids, top_lp);
}

}  // namespace kap
