// k_attn_packed.cu - attention over a pool with packed 4-bit pages (sm_103a).
//
// One warp per (query row, query head) walks its visible tokens with a running maximum and sum; a lane holds d / 32
// dims. Proposal: the entries of the request's view row. Verification: the logical pages of the block table.
#include "kap_launch.h"
#include "kap_packed.cuh"

namespace kap {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AParams {
  const __nv_bfloat16 *k, *v;
  const unsigned char *packed;
  int P16, P4, hkv, hq, R;
  const int32_t *bt;
  int max_pages;
  const int32_t *ctx_len, *seq_len;           // proposal
  ViewArgs view;                              // proposal
  const int32_t *q_offsets, *q_start;         // verification
  int rows;                                   // query rows: R, or total_q
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  float *lse;
  int *err;
};

template <int D, bool kView>
__global__ void __launch_bounds__(256) attn_kernel(const AParams p) {
  using L = PackedChunk<D>;
  constexpr int PL = D / 32;
  grid_dependency_sync();
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (wid >= static_cast<int64_t>(p.rows) * p.hq) return;
  const int row = static_cast<int>(wid / p.hq), head = static_cast<int>(wid - static_cast<int64_t>(row) * p.hq);
  const int h = head / (p.hq / p.hkv);
  int r = row, last, nent, nsel = 0, ctx = 0;
  const int32_t *ids, *lps = nullptr;
  if (kView) {
    const int vr = r * p.view.rows_per_seq + (p.view.rows_per_seq > 1 ? h : 0);
    last = p.seq_len[r] - 1;
    ctx = p.ctx_len[r];
    nent = p.view.n_entries[vr];
    nsel = p.view.n_selected[vr];
    if (nent > p.view.cap) {
      if (lane == 0) set_error(p.err, kErrCapacity);
      nent = p.view.cap;
    }
    ids = p.view.bt + static_cast<size_t>(vr) * p.view.cap;
    lps = p.view.lp + static_cast<size_t>(vr) * p.view.cap;
  } else {
    int lo = 0, hi = p.R - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.q_offsets[mid] <= row) lo = mid; else hi = mid - 1;
    }
    r = lo;
    if (row >= p.q_offsets[r + 1] || row < p.q_offsets[r]) return;
    last = p.q_start[r] + (row - p.q_offsets[r]);
    nent = last < 0 ? 0 : last / kPage + 1;
    if (nent > p.max_pages) {
      if (lane == 0) set_error(p.err, kErrPage);
      nent = p.max_pages;
    }
    ids = p.bt + static_cast<size_t>(r) * p.max_pages;
  }
  const size_t qo = (static_cast<size_t>(row) * p.hq + head) * D;
  float qv[PL], ov[PL];
  const float sc = rsqrtf(static_cast<float>(D)) * kLog2e;
#pragma unroll
  for (int k = 0; k < PL; ++k) {
    qv[k] = to_f(p.q[qo + lane + 32 * k]) * sc;
    ov[k] = 0.0f;
  }
  float mx = -INFINITY, l = 0.0f;
  for (int e = 0; e < nent; ++e) {
    const int id = ids[e], pos0 = (kView ? lps[e] : e) * kPage;
    if (id < 0 || id >= p.P16 + p.P4) {
      if (lane == 0) set_error(p.err, kErrPage);
      continue;
    }
    const unsigned char *chunk = p.packed + (static_cast<size_t>(id - p.P16) * p.hkv + h) * L::BYTES;
    const size_t o16 = (static_cast<size_t>(id) * p.hkv + h) * (kPage * D);
    for (int t = 0; t < kPage; ++t) {
      const int pos = pos0 + t;
      if (pos > last || (kView && e >= nsel && pos < ctx)) continue;
      float s = 0.0f, vv[PL];
#pragma unroll
      for (int k = 0; k < PL; ++k) {
        const int i = lane + 32 * k;
        float kk;
        if (id >= p.P16) {
          const int blk = i >> 6, at = blk * L::kBlock + t * 32 + ((i & 63) >> 1), sh = (i & 1) * 4;
          const uint32_t kp = *reinterpret_cast<const uint32_t *>(chunk + L::OFF_KPAR + (blk * kPage + t) * 4);
          const uint32_t vp = *reinterpret_cast<const uint32_t *>(chunk + L::OFF_VPAR + (blk * kPage + t) * 4);
          kk = fmaf(param_scale(kp), static_cast<float>((chunk[at] >> sh) & 15), param_low(kp));
          vv[k] = fmaf(param_scale(vp), static_cast<float>((chunk[L::OFF_V + at] >> sh) & 15), param_low(vp));
        } else {
          kk = to_f(p.k[o16 + t * D + i]);
          vv[k] = to_f(p.v[o16 + t * D + i]);
        }
        s = fmaf(qv[k], kk, s);
      }
      s = warp_sum(s);
      const float mn = fmaxf(mx, s);
      const float a = exp2f(mx - mn), w = exp2f(s - mn);
      l = l * a + w;
#pragma unroll
      for (int k = 0; k < PL; ++k) ov[k] = ov[k] * a + w * vv[k];
      mx = mn;
    }
  }
#pragma unroll
  for (int k = 0; k < PL; ++k) p.out[qo + lane + 32 * k] = from_f<__nv_bfloat16>(l != 0.0f ? ov[k] / l : 0.0f);
  if (lane == 0) {
    p.lse[static_cast<size_t>(row) * p.hq + head] = l != 0.0f ? (mx + log2f(l)) * kLn2 : -INFINITY;
    if (kView && l == 0.0f) set_error(p.err, kErrLength);
  }
}

template <bool kView>
cudaError_t launch(const PackedArgs &pa, AParams &p, const MapArgs &m, const void *q, void *out, float *lse, int *err,
                   cudaStream_t s) {
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
  p.err = err;
  const int64_t blocks = (static_cast<int64_t>(p.rows) * p.hq + 7) / 8;
  if (pa.pool.d == 128)
    return launch_pdl(attn_kernel<128, kView>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, p);
  return launch_pdl(attn_kernel<64, kView>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, p);
}

}  // namespace

size_t packed_workspace_bytes(int R, int hkv, int hq, int d, int max_q) {
  (void)R, (void)hkv, (void)hq, (void)d, (void)max_q;
  return 256;
}

cudaError_t launch_propose_packed(const PackedArgs &pa, const MapArgs &m, const ViewArgs &v, const void *q, void *out,
                                  float *lse, void *ws, int *err, cudaStream_t s) {
  (void)ws;
  AParams p{};
  p.view = v;
  p.rows = m.R;
  return launch<true>(pa, p, m, q, out, lse, err, s);
}

cudaError_t launch_verify_packed(const PackedArgs &pa, const MapArgs &m, int max_q, int total_q,
                                 const int32_t *q_offsets, const int32_t *q_start, const void *q, void *out,
                                 float *lse, void *ws, int *err, cudaStream_t s) {
  (void)ws, (void)max_q;
  AParams p{};
  p.q_offsets = q_offsets;
  p.q_start = q_start;
  p.rows = total_q;
  return launch<false>(pa, p, m, q, out, lse, err, s);
}

}  // namespace kap
