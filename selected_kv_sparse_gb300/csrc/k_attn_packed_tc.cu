// k_attn_packed_tc.cu - verification windows over packed 4-bit pages on the 5th-generation tensor cores (sm_103a), for 9
// to 64 query columns and head_dim 128.
//
// The mathematics is that of k_attn_packed.cu (bare codes in the products, parameters once per token and block); the
// tile is 8 pages = 128 tokens:
//   S_b^T[128 tok x N] = K codes of block b . q^T         (tcgen05.mma, A = fp16 codes in TMEM, lane = token)
//   O^T[128 dims x 2N] = V codes^T . [p s_0 | p s_1]^T     (A = fp16 codes in shared memory, read MN-major)
// The first 64 rows of O use the first N columns and the last 64 the others: one pass over the value codes serves both
// blocks' scales. O stays in TMEM over all tiles of a row's part; it is scaled there in the rare tile that moves a
// reference.
//
// Why here and not below 9 columns: the codes become 16-bit operands once per tile instead of once per 8 columns, and the
// logits of a token lie in one thread. Keys go to TMEM and not to shared memory, because shared memory carries the packed
// pages, the value operand (written and read once) and p already: about 116 KB a tile, 900 cycles at 128 bytes.
//
// Roles: warps 0-3 turn key codes into operands (thread = token), warps 4-7 value codes, all eight take the softmax (a
// thread has one token and half of the columns); warp 8 copies pages, warp 9 issues the MMAs. QK of tile t + 1 and PV of
// tile t run beside the softmax of the next tile.
//
// Only packed pages that every row of the window sees in full are taken. The others (16-bit pages, the window's own) are
// the business of the kernel in k_attn_packed.cu, which is launched just before, writes its records and runs beside this
// one; the last CTA to finish a row merges both kinds.
#include "kap_attn_packed.h"
#include "kap_packed.cuh"

#include <algorithm>

namespace kap {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMaxSlack = 8.0f;     // log2 units a logit may exceed its reference by
constexpr float kScaleSlack = 64.0f;  // factor a value scale may exceed its reference by
constexpr int kWorkers = 256;
constexpr int kThreads = kWorkers + 64;
constexpr int kTok = 128;
constexpr int kStages = 4;             // tiles of raw pages
constexpr int kChunk = PackedChunk<128>::BYTES;
constexpr int kMaxGrid = 160;          // CTAs, so parts of a row

template <int NP>
struct Tc {
  static constexpr int NH = NP / 2;                       // columns of a thread
  static constexpr int kRawStage = 8 * kChunk;
  static constexpr int kV = 2 * kTok * 128;               // value operand: two blocks of [128 tokens][64 dims]
  static constexpr int kP = (2 * NP > 64 ? 2 : 1) * kTok * 128;  // p operand: [128 tokens] rows of 64 columns each
  static constexpr int OFF_V = 0;
  static constexpr int OFF_P = OFF_V + 2 * kV;
  static constexpr int OFF_Q = OFF_P + 2 * kP;            // [2 blocks][NP rows][64 dims] fp16
  static constexpr int OFF_RAW = OFF_Q + 2 * NP * 128;
  static constexpr int OFF_COL = OFF_RAW + kStages * kRawStage;  // per pair of columns: cq cq q0 q0 | q1 q1 -m -m
  static constexpr int OFF_AUX = OFF_COL + NP * 16;       // [4][NP] maxima, [NP] factors, [8] scale maxima
  static constexpr int OFF_SUM = OFF_AUX + (5 * NP + 8) * 4;  // [4][NP][3] sums of a part
  static constexpr int BYTES = OFF_SUM + 12 * NP * 4 + 1024;  // room to align
  static constexpr int COL_S = 0;                         // TMEM columns: S[2][2 blocks][NP], O[NO], K[2][64]
  static constexpr int NO = 2 * NP <= 64 ? 64 : 128;      // columns of O: whole 64-column atoms of the operand
  static constexpr int COL_O = 4 * NP;
  static constexpr int COL_K = 4 * NP + NO;
  static constexpr int COLS = 4 * NP + NO + 128 <= 256 ? 256 : 512;
  static_assert(BYTES <= 227 * 1024 && 4 * NP + NO + 128 <= 512, "shared memory, TMEM");
  static_assert((kMaxGrid + kMaxRest) * 16 * 8 <= 2 * kP, "merge: maxima and sums of 16 columns lie over the p operand");
};

struct Meta {
  int valid, r, h, row, tile, first, last, nq, qoff;
  unsigned mask;  // pages of the tile that are packed and wholly visible
  int c_first, c_last;
};

__device__ __forceinline__ int atom_add_acq_rel_gpu(int *p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// fp16 inputs, fp32 accumulators; M = 128.
__device__ __forceinline__ uint32_t idesc_f16(int n, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}
// A in TMEM (lane = row, a 32-bit column = two K elements), B by descriptor.
__device__ __forceinline__ void umma_f16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float *v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Window of request r, kept inside the query array whatever the device data say.
__device__ __forceinline__ int window_of(const AttnParams &p, int r, int &qoff) {
  const int a = p.q_offsets[r], b = p.q_offsets[r + 1];
  qoff = min(max(a, 0), p.total_q);
  return min(max(min(b, p.total_q) - qoff, 0), p.max_q);
}
// Tiles of a row of request r: those of the pages that its first window row sees in full, one at least.
__device__ __forceinline__ int tiles_of(const AttnParams &p, int r) {
  int qoff;
  if (window_of(p, r, qoff) <= 0) return 0;
  const int64_t full = max((static_cast<int64_t>(p.q_start[r]) + 1) / kPage, static_cast<int64_t>(0));
  return max(static_cast<int>((min(full, static_cast<int64_t>(p.max_pages)) + 7) / 8), 1);
}

template <int NP>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const AttnParams p) {
  using T = Tc<NP>;
  constexpr int NH = T::NH;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  float *colp = reinterpret_cast<float *>(sm + T::OFF_COL);
  float *aux_max = reinterpret_cast<float *>(sm + T::OFF_AUX), *aux_f = aux_max + 4 * NP, *aux_sv = aux_f + NP;
  float *sums = reinterpret_cast<float *>(sm + T::OFF_SUM);
  __shared__ uint64_t s_bars[2 * kStages + 13];
  __shared__ Meta s_meta[kStages];
  __shared__ int64_t s_scan[kThreads / 32], s_total, s_base;
  __shared__ int s_req, s_abort, s_flag, s_or[3];
  __shared__ uint32_t s_tmem;
  uint64_t *raw_full = s_bars, *raw_free = raw_full + kStages, *k_ready = raw_free + kStages, *v_ready = k_ready + 2,
           *s_full = v_ready + 2, *p_ready = s_full + 2, *o_done = p_ready + 2, *q_ready = o_done + 2, *sync_bar = q_ready + 1, *drained = sync_bar + 1;
  volatile int *abort_flag = &s_abort;
  auto aborted = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0) != 0; };  // alike for a warp's lanes
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.hq / p.hkv;

  // No dependency wait here: what is read before the merge was written before the kernel just ahead of this one (the one
  // that takes the other pages), and that one has waited for its own predecessor.
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kStages; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_free[i], 9);  // 8 workers, the MMA warp
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_ready[i], 4);
      mbar_init(&v_ready[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 8);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(q_ready, 8);
    mbar_init(sync_bar, 8);
    mbar_init(drained, 1);
    s_or[0] = s_or[1] = s_or[2] = 0;
    fence_barrier_init();
  }
  // ---- this CTA's share of the line of tiles, and the request that it starts in
  int64_t total = 0, incl = 0, own = 0;
  for (int base = 0; base < p.R; base += kThreads) {
    const int r = base + tid;
    own = r < p.R ? static_cast<int64_t>(tiles_of(p, r)) * p.hkv : 0;
    incl = block_inclusive_scan<int64_t>(own, s_scan);
    if (tid == kThreads - 1) s_total = incl;
    __syncthreads();
    total += s_total;
    __syncthreads();
  }
  const int64_t share = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(1));
  const int64_t x0 = share * blockIdx.x, x1 = min(x0 + share, total);
  if (x0 >= x1) {
    grid_dependency_sync();
    return;
  }
  if (p.R <= kThreads) {
    if (incl - own <= x0 && x0 < incl) s_req = tid, s_base = incl - own;
  } else {
    int64_t before = 0;
    for (int base = 0; base < p.R; base += kThreads) {
      const int r = base + tid;
      const int64_t n = r < p.R ? static_cast<int64_t>(tiles_of(p, r)) * p.hkv : 0;
      const int64_t upto = before + block_inclusive_scan<int64_t>(n, s_scan);
      if (upto - n <= x0 && x0 < upto) s_req = r, s_base = upto - n;
      if (tid == kThreads - 1) s_total = upto;
      __syncthreads();
      before = s_total;
      __syncthreads();
      if (before > x0) break;
    }
  }
  if (warp == 9) {
    tmem_alloc(&s_tmem, T::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == 8) {
    // ============================================================================================== pages
    int r = s_req, nt = tiles_of(p, r), qoff = 0, nq = window_of(p, r, qoff);
    int64_t base = s_base;
    const uint64_t pol = l2_evict_first_policy();
    int t = 0;
    for (int64_t x = x0;; ++x, ++t) {
      const int st = t % kStages;
      Meta m;
      m.valid = x < x1 && !aborted();
      int id = -1;
      bool ok = false;
      if (m.valid) {
        while (x >= base + static_cast<int64_t>(nt) * p.hkv) {
          base += static_cast<int64_t>(nt) * p.hkv;
          nt = tiles_of(p, ++r);
          nq = window_of(p, r, qoff);
        }
        const int in = static_cast<int>(x - base);
        m.r = r;
        m.h = in / nt;
        m.tile = in - m.h * nt;
        m.row = r * p.hkv + m.h;
        m.first = x == x0 || m.tile == 0;
        m.last = x + 1 == x1 || m.tile + 1 == nt;
        m.nq = nq;
        m.qoff = qoff;
        const int64_t rb = x - m.tile;
        m.c_first = static_cast<int>(rb / share);
        m.c_last = static_cast<int>((rb + nt - 1) / share);
        const int page = m.tile * 8 + lane;
        if (lane < 8 && page < p.max_pages && page * kPage + kPage - 1 <= p.q_start[r])
          id = p.bt[static_cast<size_t>(r) * p.max_pages + page];
        ok = id >= p.P16 && id < p.P16 + p.P4;
      }
      m.mask = __ballot_sync(0xffffffffu, ok);
      if (t >= kStages && !__all_sync(0xffffffffu, mbar_wait(&raw_free[st], ((t / kStages) - 1) & 1, p.err))) {
        *abort_flag = 1;
        break;
      }
      if (lane == 0) {
        s_meta[st] = m;
        mbar_arrive_expect_tx(&raw_full[st], __popc(m.mask) * kChunk);
      }
      __syncwarp();
      if (ok)
        bulk_g2s_stream(sm + T::OFF_RAW + st * T::kRawStage + lane * kChunk,
                        p.packed + (static_cast<size_t>(id - p.P16) * p.hkv + m.h) * kChunk, kChunk, &raw_full[st], pol);
      if (!m.valid) break;
    }
    // copies in flight after an abort are waited for, with a limit
    if (*abort_flag && lane == 0)
      for (int u = max(0, t - kStages); u < t; ++u) mbar_wait(&raw_full[u % kStages], (u / kStages) & 1, nullptr);
  } else if (warp == 9) {
    // ============================================================================================== MMAs
    if (lane == 0) {
      const uint32_t idqk = idesc_f16(NP, 0, 0), idpv = idesc_f16(T::NO, 1, 1);
      const uint32_t qb = smem_u32(sm + T::OFF_Q);
      int segs = 0;
      bool first_prev = true, ok = true;
      for (int t = 0; ok; ++t) {
        bool valid = false, first = false;
        ok = mbar_wait(&raw_full[t % kStages], (t / kStages) & 1, p.err);  // the tile's description
        if (ok) {
          valid = s_meta[t % kStages].valid;
          first = s_meta[t % kStages].first;
          if (valid) mbar_arrive(&raw_free[t % kStages]);
        }
        const int b = t & 1;
        auto qk = [&]() {
          ok = mbar_wait(&k_ready[b], (t >> 1) & 1, p.err);
          if (ok && first) ok = mbar_wait(q_ready, segs++ & 1, p.err);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_tmem_a(tmem + T::COL_S + b * 2 * NP + blk * NP, tmem + T::COL_K + b * 64 + blk * 32 + kk * 8,
                              smem_desc(qb + blk * NP * 128 + kk * 32, 16, 1024, 2), idqk, kk > 0 ? 1u : 0u);
          umma_commit(&s_full[b]);
        };
        // the next tile's logits ahead of this one's values, but for a part's first tile: its queries are written only
        // when the part before is finished
        if (ok && valid && !first) qk();
        if (ok && t > 0) {  // PV of the tile before
          const int c = (t - 1) & 1;
          ok = mbar_wait(&v_ready[c], ((t - 1) >> 1) & 1, p.err) && mbar_wait(&p_ready[c], ((t - 1) >> 1) & 1, p.err);
          if (ok) {
            tc_fence_after();
            const uint32_t vb = smem_u32(sm + T::OFF_V + c * T::kV), pb = smem_u32(sm + T::OFF_P + c * T::kP);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_bf16(tmem + T::COL_O, smem_desc(vb + kk * 2048, kTok * 128, 1024, 2),
                        smem_desc(pb + kk * 2048, kTok * 128, 1024, 2), idpv, kk > 0 || !first_prev ? 1u : 0u);
            umma_commit(&o_done[c]);
          }
        }
        if (ok && valid && first) qk();
        first_prev = first;
        if (!valid) break;
      }
      if (!ok) *abort_flag = 1;
      umma_commit(drained);  // nothing of this CTA is in the tensor pipe when its TMEM is freed
      mbar_wait(drained, 0, p.err);
    }
    __syncwarp();
  } else {
    // ============================================================================================== workers
    const int quad = warp & 3, hf = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const int tok = quad * 32 + lane;
    const float qk = rsqrtf(128.0f) * kLog2e;
    F2 lsum[NH / 2], lv0[NH / 2], lv1[NH / 2];
    float inv_e = 1.0f, sv_limit = 0.0f;
    bool fresh = true;  // no token of the part seen so far: every column sees the same ones
    auto wait = [&](uint64_t *bar, int parity) {
      if (aborted()) return;
      if (!__all_sync(0xffffffffu, mbar_wait(bar, parity, p.err))) *abort_flag = 1;
    };
    // Barriers among the eight workers. They are bounded waits like all others: a warp that gave up leaves its loop, and
    // the others follow at their next wait.
    volatile int *or_slot = s_or;
    int syncs = 0, ors = 0;
    auto workers_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(sync_bar);
      wait(sync_bar, syncs++ & 1);
    };
    auto workers_or = [&](bool v) {
      const int k = ors++ % 3;
      if (__any_sync(0xffffffffu, v) && lane == 0) or_slot[k] = 1;
      workers_sync();
      const bool r = or_slot[k] != 0;
      if (tid == 0) or_slot[(k + 2) % 3] = 0;  // read by all before this barrier, used again after the next
      return r;
    };
    // keys or values of tile t to operands; the tile's description and this token's parameters into registers
    Meta m, nm;
    uint32_t kp0 = 0, kp1 = 0, vp0 = 0, vp1 = 0, nk0 = 0, nk1 = 0, nv0 = 0, nv1 = 0;
    auto take = [&](int t) {
      const int st = t % kStages, b = t & 1;
      const unsigned char *raw = sm + T::OFF_RAW + st * T::kRawStage;
      wait(&raw_full[st], (t / kStages) & 1);
      nm = s_meta[st];
      if (aborted()) nm.valid = 0;
      if (!nm.valid) return;
      const unsigned char *mine = raw + (tok >> 4) * kChunk;
      const int o = tok & 15;
      nk0 = *reinterpret_cast<const uint32_t *>(mine + PackedChunk<128>::OFF_KPAR + o * 4);
      nk1 = *reinterpret_cast<const uint32_t *>(mine + PackedChunk<128>::OFF_KPAR + 64 + o * 4);
      nv0 = *reinterpret_cast<const uint32_t *>(mine + PackedChunk<128>::OFF_VPAR + o * 4);
      nv1 = *reinterpret_cast<const uint32_t *>(mine + PackedChunk<128>::OFF_VPAR + 64 + o * 4);
      if (hf == 0) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          const uint4 a = *reinterpret_cast<const uint4 *>(mine + blk * 512 + o * 32);
          const uint4 c = *reinterpret_cast<const uint4 *>(mine + blk * 512 + o * 32 + 16);
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
          uint32_t out[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            out[4 * i] = w[i] & 0x000f000fu;
            out[4 * i + 1] = w[i] & 0x00f000f0u;
            out[4 * i + 2] = (w[i] >> 8) & 0x000f000fu;
            out[4 * i + 3] = (w[i] >> 8) & 0x00f000f0u;
          }
          tmem_st32(tmem + T::COL_K + b * 64 + blk * 32 + lane_base, out);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&k_ready[b]);
          mbar_arrive(&raw_free[st]);
        }
      } else {
        if (t >= 2) wait(&o_done[b], ((t >> 1) - 1) & 1);  // the value operand's last reader
        unsigned char *vd = sm + T::OFF_V + b * T::kV;
        const int wd = lane & 7;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {  // 4 tokens of a block at a time: 8 lanes write a token's 128 bytes
          const int blk = i >> 3, tk = quad * 32 + (i & 7) * 4 + (lane >> 3);
          const uint32_t w = *reinterpret_cast<const uint32_t *>(raw + (tk >> 4) * kChunk + PackedChunk<128>::OFF_V +
                                                                 blk * 512 + (tk & 15) * 32 + wd * 4);
          *reinterpret_cast<uint4 *>(vd + blk * (kTok * 128) + tk * 128 + ((wd ^ (tk & 7)) << 4)) =
              make_uint4(w & 0x000f000fu, w & 0x00f000f0u, (w >> 8) & 0x000f000fu, (w >> 8) & 0x00f000f0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&v_ready[b]);
          mbar_arrive(&raw_free[st]);
        }
      }
    };
    take(0);
    for (int t = 0;; ++t) {
      m = nm;
      kp0 = nk0, kp1 = nk1, vp0 = nv0, vp1 = nv1;
      if (!m.valid || aborted()) break;
      const int b = t & 1;
      const int M = G * m.nq;
      if (m.first) {
        // ---- queries of the row: fp16 operands (K-major, 128-byte swizzle) and the columns' constants
        workers_sync();
        for (int i = tid; i < NP * 16; i += kWorkers) {
          const int c = i >> 4, piece = i & 15;
          uint4 raw = make_uint4(0, 0, 0, 0);
          if (c < M) {
            const int w = c / G, a = c - w * G;
            raw = *reinterpret_cast<const uint4 *>(p.q + (static_cast<size_t>(m.qoff + w) * p.hq + m.h * G + a) * 128 + piece * 8);
          }
          float v[8];
          Vec16<__nv_bfloat16>::unpack(raw, v);
          float mx = 0.0f, sum = 0.0f;
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            mx = fmaxf(mx, fabsf(v[z]));
            sum += v[z];
          }
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll
          for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          // largest magnitude to [2^14, 2^15): every bf16 down to 2^-24 of it is exact in fp16, a sixteenth too
          const int e = static_cast<int>((__float_as_uint(mx) >> 23) & 255);
          const int sh = e == 0 || e == 255 ? 0 : min(141 - e, 126);
          const float sc = __uint_as_float(static_cast<uint32_t>(127 + max(sh, -126)) << 23), s16 = sc * 0.0625f;
          float *cp = colp + (c >> 1) * 8 + (c & 1);
          if (piece == 0) {
            cp[0] = qk * 0x1p24f / sc;
            cp[6] = 0.0f;
          }
          if ((piece & 7) == 0) cp[2 + 2 * (piece >> 3)] = sum * qk;
          const int blk = piece >> 3, wd = piece & 7;
          *reinterpret_cast<uint4 *>(sm + T::OFF_Q + blk * NP * 128 + c * 128 + ((wd ^ (c & 7)) << 4)) =
              make_uint4(pack_f16(v[0] * sc, v[4] * sc), pack_f16(v[1] * s16, v[5] * s16), pack_f16(v[2] * sc, v[6] * sc),
                         pack_f16(v[3] * s16, v[7] * s16));
        }
        fence_proxy_async_smem();
        workers_sync();
        if (lane == 0) mbar_arrive(q_ready);
#pragma unroll
        for (int j = 0; j < NH / 2; ++j) lsum[j] = lv0[j] = lv1[j] = f2(0.0f, 0.0f);
        inv_e = 1.0f;
        sv_limit = 0.0f;
        fresh = true;
      }
      if (hf == 0) take(t + 1);
      // ---- logits of this token, over the columns' references
      wait(&s_full[b], (t >> 1) & 1);
      tc_fence_after();
      const bool seen = (m.mask >> (tok >> 4)) & 1u;
      if (!seen) vp0 = vp1 = 0u;
      F2 d[NH / 2];
      float over = -INFINITY;
      {
        const float4 *cp4 = reinterpret_cast<const float4 *>(colp) + hf * NH;
        const float fk0 = param_scale(kp0), fk1 = param_scale(kp1), fl0 = param_low(kp0), fl1 = param_low(kp1);
        const F2 sk0 = f2(fk0, fk0), sk1 = f2(fk1, fk1), lo0 = f2(fl0, fl0), lo1 = f2(fl1, fl1);
#pragma unroll
        for (int g = 0; g < NH / 8; ++g) {
          float s0[8], s1[8];
          const uint32_t at = tmem + T::COL_S + b * 2 * NP + hf * NH + g * 8 + lane_base;
          tmem_ld8(at, s0);
          tmem_ld8(at + NP, s1);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 ca = cp4[(g * 4 + j) * 2], cb = cp4[(g * 4 + j) * 2 + 1];
            const F2 a = fma2(f2(s1[2 * j], s1[2 * j + 1]), sk1, mul2(f2(s0[2 * j], s0[2 * j + 1]), sk0));
            const F2 l = fma2(lo1, f2(cb.x, cb.y), fma2(lo0, f2(ca.z, ca.w), f2(cb.z, cb.w)));
            float x, y;
            split(fma2(a, f2(ca.x, ca.y), l), x, y);
            if (!seen) x = y = -INFINITY;
            d[g * 4 + j] = f2(x, y);
            over = fmaxf(over, fmaxf(x, y));
          }
        }
      }
      tc_fence_before();
      float sv0 = param_scale(vp0), sv1 = param_scale(vp1);
      const float svmax = fmaxf(fmaxf(sv0, sv1), 0.0f);
      if (workers_or(over > kMaxSlack || svmax > sv_limit || (fresh && seen))) {
        // ---- references moved: column maxima over the tile's tokens, then the factors of what is summed so far
#pragma unroll
        for (int j = 0; j < NH / 2; ++j) {
          float x, y;
          split(d[j], x, y);
          x = warp_max(x);
          y = warp_max(y);
          if (lane == 0) {
            aux_max[quad * NP + hf * NH + 2 * j] = x;
            aux_max[quad * NP + hf * NH + 2 * j + 1] = y;
          }
        }
        const float wsv = warp_max(svmax);
        if (lane == 0) aux_sv[warp] = wsv;
        workers_sync();
        float mx = 0.0f, ratio = 1.0f;
        for (int w = 0; w < 4; ++w) mx = fmaxf(mx, aux_sv[w]);
        if (mx > sv_limit) {
          const float ie = 1.0f / fmaxf(__uint_as_float(__float_as_uint(mx) & 0x7f800000u), 0x1p-100f);
          ratio = ie / inv_e;
          inv_e = ie;
          sv_limit = kScaleSlack / ie;
        }
        if (tid < NP) {
          // by how much the reference rises; the first tokens set it, up or down
          float up = fmaxf(fmaxf(aux_max[tid], aux_max[NP + tid]), fmaxf(aux_max[2 * NP + tid], aux_max[3 * NP + tid]));
          if (fresh ? !(up > kNoMax) : !(up > 0.0f)) up = 0.0f;
          float *cp = colp + (tid >> 1) * 8 + (tid & 1);
          const float old = -cp[6], now = old + up;
          cp[6] = -now;
          aux_f[tid] = now - old;
        }
        workers_sync();
#pragma unroll
        for (int j = 0; j < NH / 2; ++j) {
          const float ux = aux_f[hf * NH + 2 * j], uy = aux_f[hf * NH + 2 * j + 1];
          d[j] = add2(d[j], f2(-ux, -uy));
          if (fresh) continue;
          const F2 f = f2(fast_exp2(-ux), fast_exp2(-uy));
          lsum[j] = mul2(lsum[j], f);
          lv0[j] = mul2(lv0[j], f);
          lv1[j] = mul2(lv1[j], f);
        }
        if (!fresh) {
          wait(&o_done[b ^ 1], ((t - 1) >> 1) & 1);  // O as of the tile before
          tc_fence_after();
          // O rows of this warp's lanes, half of the columns of either block
#pragma unroll
          for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int g = 0; g < NH / 8; ++g) {
              float o[8];
              const uint32_t at = tmem + T::COL_O + blk * NP + hf * NH + g * 8 + lane_base;
              tmem_ld8(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int z = 0; z < 8; ++z) o[z] *= fast_exp2(-aux_f[hf * NH + g * 8 + z]) * ratio;
              tmem_st8(at, o);
            }
          tmem_wait_st();
          tc_fence_before();
        }
        fresh = false;
      }
      // ---- probabilities; p times the value scales as the second product's operand (MN-major rows, 128-byte swizzle)
      if (t >= 2) wait(&o_done[b], ((t >> 1) - 1) & 1);  // its last reader
      {
        const float e0 = sv0 * inv_e, e1 = sv1 * inv_e, l0 = param_low(vp0), l1 = param_low(vp1);
        const F2 x0 = f2(e0, e0), x1w = f2(e1, e1), w0 = f2(l0, l0), w1 = f2(l1, l1);
        unsigned char *pd = sm + T::OFF_P + b * T::kP + tok * 128;
#pragma unroll
        for (int g = 0; g < NH / 8; ++g) {
          uint32_t h0[4], h1[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x, y;
            split(d[g * 4 + j], x, y);
            const F2 pr = f2(fast_exp2(x), fast_exp2(y));
            lsum[g * 4 + j] = add2(lsum[g * 4 + j], pr);
            lv0[g * 4 + j] = fma2(pr, w0, lv0[g * 4 + j]);
            lv1[g * 4 + j] = fma2(pr, w1, lv1[g * 4 + j]);
            split(mul2(pr, x0), x, y);
            h0[j] = pack_f16(x, y);
            split(mul2(pr, x1w), x, y);
            h1[j] = pack_f16(x, y);
          }
          const int c0 = (hf * NH) / 8 + g, c1 = (NP + hf * NH) / 8 + g;  // 16-byte chunks of the token's row
          *reinterpret_cast<uint4 *>(pd + (c0 >> 3) * (kTok * 128) + (((c0 & 7) ^ (tok & 7)) << 4)) =
              make_uint4(h0[0], h0[1], h0[2], h0[3]);
          *reinterpret_cast<uint4 *>(pd + (c1 >> 3) * (kTok * 128) + (((c1 & 7) ^ (tok & 7)) << 4)) =
              make_uint4(h1[0], h1[1], h1[2], h1[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[b]);
      if (hf == 1) take(t + 1);

      if (m.last) {
        // ---- the part's sums over tokens, then its record: O in its own unit, and what the lowest values add
#pragma unroll
        for (int j = 0; j < NH / 2; ++j) {
          float v[6];
          split(lsum[j], v[0], v[3]);
          split(lv0[j], v[1], v[4]);
          split(lv1[j], v[2], v[5]);
#pragma unroll
          for (int z = 0; z < 6; ++z) v[z] = warp_sum(v[z]);
          if (lane < 6) {
            float o = v[0];
#pragma unroll
            for (int z = 1; z < 6; ++z) o = lane == z ? v[z] : o;
            sums[(quad * NP + hf * NH + 2 * j + lane / 3) * 3 + lane % 3] = o;
          }
        }
        wait(&o_done[b], (t >> 1) & 1);
        tc_fence_after();
        workers_sync();
        const size_t slot = static_cast<size_t>(blockIdx.x) + m.row;
        const int blk = quad >> 1;                  // rows below 64 are dims of the first block
        const int j8 = tok & 7, perm = ((j8 & 1) << 2) | (j8 >> 1);
        const float unit = ((j8 & 2) ? 0x1p20f : 0x1p24f) / inv_e;
#pragma unroll
        for (int g = 0; g < NH / 8; ++g) {
          float o[8];
          tmem_ld8(tmem + T::COL_O + blk * NP + hf * NH + g * 8 + lane_base, o);
          tmem_wait_ld();
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const int col = hf * NH + g * 8 + z;
            if (col >= M) continue;
            float l = 0.0f, v = 0.0f;
            for (int q = 0; q < 4; ++q) {
              l += sums[(q * NP + col) * 3];
              v += sums[(q * NP + col) * 3 + 1 + blk];
            }
            __stcg(p.part + (slot * p.ncol + col) * 128 + (tok & ~7) + perm, fmaf(o[z], unit, v));
            if (tok == 0) __stcg(&p.ml[slot * p.ncol + col], make_float2(fresh ? kNoMax : -colp[(col >> 1) * 8 + 6 + (col & 1)], l));
          }
        }
        tc_fence_before();
        // the other kernel's records are complete from here on; its successor may start
        grid_dependency_wait();
        workers_sync();
        if (tid == 0) {
          const int old = atom_add_acq_rel_gpu(&p.counters[m.row], 1);
          s_flag = old == m.c_last - m.c_first;
          if (s_flag) p.counters[m.row] = 0;  // left at zero for the next call
        }
        workers_sync();
        if (s_flag && !aborted()) {
          // parts of this kernel in the slots from c_first + row, the other's behind rest_slot; 16 columns at a time: the
          // weights, then every thread sums 8 dims in the parts' order
          float2 *area = reinterpret_cast<float2 *>(sm + T::OFF_P);
          const int mine = m.c_last - m.c_first + 1, parts = mine + p.rest;
          const size_t slot0 = static_cast<size_t>(m.c_first) + m.row, rest0 = p.rest_slot + static_cast<size_t>(m.row) * p.rest;
          for (int c0 = 0; c0 < M; c0 += 16) {
            const int n = min(16, M - c0);
            for (int i = tid; i < parts * 16; i += kWorkers) {
              const int k = i >> 4, c = i & 15;
              if (c < n) area[i] = __ldcg(&p.ml[(k < mine ? slot0 + k : rest0 + (k - mine)) * p.ncol + c0 + c]);
            }
            workers_sync();
            if (tid < n) {
              float mx = kNoMax, l = 0.0f;
              for (int k = 0; k < parts; ++k) mx = fmaxf(mx, area[k * 16 + tid].x);
              for (int k = 0; k < parts; ++k) {
                const float2 z = area[k * 16 + tid];
                const float f = fast_exp2(z.x - mx);
                l = fmaf(z.y, f, l);
                area[k * 16 + tid].x = f;
              }
              area[tid].y = l != 0.0f ? 1.0f / l : 0.0f;  // the first part's pair: the factor of the whole column
              const int col = c0 + tid, w = col / G;
              p.lse[static_cast<size_t>(m.qoff + w) * p.hq + m.h * G + (col - w * G)] =
                  l != 0.0f ? (mx + log2f(l)) * kLn2 : -INFINITY;
            }
            workers_sync();
            if ((tid >> 4) < n) {
              const int c = tid >> 4, col = c0 + c, d0 = (tid & 15) * 8, w = col / G;
              float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
              for (int k = 0; k < parts; ++k) {
                const float *rec = p.part + ((k < mine ? slot0 + k : rest0 + (k - mine)) * p.ncol + col) * 128 + d0;
                const float4 a = __ldcg(reinterpret_cast<const float4 *>(rec));
                const float4 e = __ldcg(reinterpret_cast<const float4 *>(rec + 4));
                const float f = area[k * 16 + c].x;
                v[0] = fmaf(a.x, f, v[0]), v[1] = fmaf(a.y, f, v[1]), v[2] = fmaf(a.z, f, v[2]), v[3] = fmaf(a.w, f, v[3]);
                v[4] = fmaf(e.x, f, v[4]), v[5] = fmaf(e.y, f, v[5]), v[6] = fmaf(e.z, f, v[6]), v[7] = fmaf(e.w, f, v[7]);
              }
#pragma unroll
              for (int z = 0; z < 8; ++z) v[z] *= area[c].y;
              *reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(m.qoff + w) * p.hq + m.h * G + (col - w * G)) * 128 + d0) =
                  Vec16<__nv_bfloat16>::pack(v);
            }
            workers_sync();
          }
        }
        workers_sync();
      }
    }
  }
  __syncthreads();
  grid_dependency_sync();
  if (warp == 9) tmem_dealloc(tmem, T::COLS);
}

template <int NP>
cudaError_t launch(const AttnParams &p, cudaStream_t s) {
  using T = Tc<NP>;
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev & 63]) {
    e = cudaFuncSetAttribute(attn_tc_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::BYTES);
    if (e != cudaSuccess) return e;
    ready[dev & 63] = true;
  }
  return launch_pdl(attn_tc_kernel<NP>, dim3(std::min(device_sm_count(), kMaxGrid)), dim3(kThreads), T::BYTES, s, p);
}

}  // namespace

cudaError_t launch_attn_packed_tc(const AttnParams &p, cudaStream_t s) {
  if (p.ncol <= 16) return launch<16>(p, s);
  if (p.ncol <= 32) return launch<32>(p, s);
  if (p.ncol <= 48) return launch<48>(p, s);
  return launch<64>(p, s);
}

}  // namespace kap
