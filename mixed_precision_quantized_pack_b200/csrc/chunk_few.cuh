// Chunk attention with up to 24 query rows of a kv head (one or a few new tokens), and with any number
// over a cache with a side code, 16 at a time: the one-token
// decode kernel's design (decode_mma.cuh) with a query row per MMA column.
//
// One CTA = 4 warps = one split of one (b, kv head): splits [0, splits_q) cover whole key groups of
// the quantized prefix, the others the fp16 list followed by the new tokens.  Units (key groups, or
// tiles of 16 fp16 rows) go round-robin to the warps through a ring of bulk-copied shared-memory
// stages.  Scores: mma.m16n8k16 with 16 tokens on M, 8 query rows on N (one to three such n-tiles);
// key codes are masked in place as fp16 subnormals (one AND per two codes), the per-channel key
// scales are folded into the query once per group and the zero points add one MMA per k-step.
// p.V: channels on M, tokens on K, query rows on N, weights p_j * s_{j,g} moved to the B layout with
// movmatrix, value codes as centred subnormals (code - 2^(bits-1): their fp32 accumulators stay near
// zero in a long context).
//
// Up to four rows, query products and weights take two columns each, their two fp16 halves, as in the
// decode kernel (error 2e-4 against 64 bits, the output's own rounding).  From five rows on they are
// rounded to fp16 once (10e-4): twice the rows for the same work.  Sums, maxima and
// accumulators are fp32.  Bound: instruction issue (a code unpack per 8 to 24 rows), with the
// cache's bytes not far below; the tcgen05 kernels decode to shared memory first, which few rows do
// not pay for (over 32 x 32k, 16 rows 0.42 ms here and 0.59 there, 24 rows 0.57 and 0.71; K2V2 over
// 16 x 16k, 24 rows 0.17 and 0.22; K4V4 0.18 and 0.20).  Groups of 32 with 4-bit keys and 2-bit values
// are about even at 17 to 24 rows (20 rows, 8 kv heads: 4 x 32k 111 us here and 131 there, 12 x 2k 46
// and 66, 8 x 16k 124 and 125; 16 x 16k 221 and 214, 12 x 8k 133 and 113, 16 x 2k 66 and 55).  A fourth
// n-tile spills 900 bytes a thread (32 rows over 32 x 32k 1.00 ms, 0.72 there).
#pragma once

#include "decode_mma.cuh"
#include "seq_ops.cuh"

namespace kvq {
namespace few {

using mma::kCtasPerSm;
using mma::kDV;
using mma::kMaxRing;
using mma::kThreads;
using mma::kWaitLimitNs;
using mma::kWarps;

// Shared memory of one CTA: the queries for the zero-point MMA and scaled for the score MMA (each
// u32 [NT][2*KSTEPS][32 lanes]), then barriers, copy counters, unit tags, failure flag, pages, and
// the ring of stages.
template <int KSTEPS, int NT, int SR>
struct Smem {
  static constexpr int kQb = 0;
  static constexpr int kQf = kQb + NT * 2 * KSTEPS * 32 * 4;
  static constexpr int kBars = kQf + NT * 2 * KSTEPS * 32 * 4;
  static constexpr int kIssued = kBars + kMaxRing * 8;
  static constexpr int kTag = kIssued + kMaxRing * 4;
  static constexpr int kFail = kTag + kMaxRing * 4;
  static constexpr int kPage = kFail + 16;
  static constexpr int kQt = kPage + 16;                     // U_h^T q: fp32 [8 NT rows][SR]
  static constexpr int kStages = kBars + (SR ? 256 + 8 * NT * SR * 4 : 256);
  static_assert(kQt - kBars <= 256 && kStages % 128 == 0, "header");
};

template <int KB, int VB, int DK, int GV, int GK, int SR, int SQ, int ROWS>
struct Rings {
  static constexpr int NT = (ROWS + 7) / 8;
  // four CTAs an SM with one n-tile, two with two or three: their accumulators spill at 168 registers
  static constexpr int CTAS = NT == 1 ? 4 : 2;
  static constexpr int AVAIL = 233472 / CTAS - 1024;
  static constexpr int HDR = Smem<DK / 16, NT, SR>::kStages;
  static constexpr int STAGE_Q = mma::quant_stage_bytes<KB, VB, DK, GV, GK, SR, SQ>();
  static constexpr int STAGE_F = mma::raw_stage_bytes<DK>();
  static constexpr int RING_Q = mma::ring_for(AVAIL - HDR, STAGE_Q, mma::kMinRing);
  static constexpr int RING_F = mma::ring_for(AVAIL - HDR, STAGE_F, kWarps);
  static constexpr int MERGE = kWarps * ROWS * (kDV + 2) * 4;
  static constexpr int STAGES = RING_Q * STAGE_Q > RING_F * STAGE_F ? RING_Q * STAGE_Q : RING_F * STAGE_F;
  static constexpr int BYTES = HDR + (STAGES > MERGE ? STAGES : MERGE);
};

// Two weights as the fp16 pair of a B register: those of two rows, or one's halves.
template <bool HALVES>
__device__ __forceinline__ uint32_t weights(float w0, float w1) {
  if constexpr (HALVES) {
    const float hi = __half2float(__float2half_rn(w0));
    return ptx::h2_as_u32(__floats2half2_rn(hi, w0 - hi));
  }
  return ptx::h2_as_u32(__floats2half2_rn(w0, w1));
}

template <int KB, int VB, int DK, int GV, int GK, int SR, int SQ, int ROWS>
__global__ void __launch_bounds__(kThreads, Rings<KB, VB, DK, GV, GK, SR, SQ, ROWS>::CTAS)
chunk_few_kernel(const __grid_constant__ Dims d, const __grid_constant__ CacheBufs cb,
                 const __grid_constant__ ChunkArgs a) {
  using G = mma::Quant<KB, VB, DK, GV>;
  using R = mma::Raw<DK>;
  constexpr int KSTEPS = DK / 16;
  using RG = Rings<KB, VB, DK, GV, GK, SR, SQ, ROWS>;
  constexpr int NT = RG::NT;
  constexpr bool HALVES = ROWS == 4;         // columns 2r, 2r + 1: the two fp16 halves of row r
  constexpr int RPT = HALVES ? 1 : 2;        // a thread's query rows per n-tile
  using SM = Smem<KSTEPS, NT, SR>;
  using Z = mma::Side<SR, SQ>;
  extern __shared__ __align__(128) unsigned char smem[];

  const int split = blockIdx.x % a.splits, rb = blockIdx.x / a.splits * ROWS;   // the block's first query row
  const int h = blockIdx.y, b = blockIdx.z;
  const int bh = b * d.Hkv + h;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qi = lane & 3;          // C columns 2qi, 2qi+1
  const int qr = lane >> 2;         // A rows qr, qr+8; B column qr
  const bool low = HALVES && (qr & 1) != 0;      // the B column holds low halves
  const SeqNew sw = seq_new(a.seq, b, d.log_retain);
  if (sw.n == 0) return;
  const int n_rows = d.n_rep * a.T;
  // the new tokens that some row of the block may see; none of its rows may be valid
  int n_vis = sw.n;
  {
    const int r1 = min(rb + ROWS, n_rows) - 1;
    if (rb / a.T == r1 / a.T) {                 // rows of one head: tokens rb % T to r1 % T
      if (rb % a.T >= sw.n) return;
      if (!a.mask) n_vis = min(n_vis, r1 % a.T + 1);
    }
  }

  uint32_t* sm_qb = reinterpret_cast<uint32_t*>(smem + SM::kQb);
  uint32_t* sm_qf = reinterpret_cast<uint32_t*>(smem + SM::kQf);
  int* sm_issued = reinterpret_cast<int*>(smem + SM::kIssued);
  volatile int* sm_tag = reinterpret_cast<volatile int*>(smem + SM::kTag);
  int* sm_fail = reinterpret_cast<int*>(smem + SM::kFail);
  const uint32_t bar0 = ptx::smem_addr(smem + SM::kBars);
  unsigned char* stages = smem + SM::kStages;
  const uint32_t stages_s = ptx::smem_addr(stages);

  const bool quant = split < a.splits_q;
  const int ring = quant ? RG::RING_Q : RG::RING_F;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ring; ++s) {
      ptx::mbar_init(bar0 + 8 * s, 1);
      sm_issued[s] = 0;
      sm_tag[s] = -1;
    }
    *sm_fail = 0;
    ptx::fence_barrier_init();
  }
  // the query row of this thread's B column, per n-tile (rows that are not there, or behind the
  // sequence's new tokens, are zero)
  const __half* qrow[NT];
  bool qok[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = rb + 8 * nt + (HALVES ? qr >> 1 : qr);
    qok[nt] = r < n_rows && r % a.T < sw.n;
    qrow[nt] = a.q + (static_cast<size_t>(bh) * n_rows + (qok[nt] ? r : 0)) * DK;
  }

  // ---------------- work list of this CTA ----------------
  const int n_old = sw.n_ret + sw.L - sw.Q, n_list = n_old + n_vis;    // the fp16 list, then the new tokens
  int unit_begin, unit_end, list_begin = 0, list_end = 0;
  if (quant) {
    const long long groups = sw.Q / GK;
    unit_begin = static_cast<int>(split * groups / a.splits_q);
    unit_end = static_cast<int>((split + 1) * groups / a.splits_q);
  } else {
    const int f = split - a.splits_q, nf = a.splits - a.splits_q;
    list_begin = static_cast<int>(static_cast<long long>(f) * n_list / nf);
    list_end = static_cast<int>(static_cast<long long>(f + 1) * n_list / nf);
    unit_begin = 0;
    unit_end = (list_end - list_begin + 15) / 16;
  }
  const int n_units = unit_end - unit_begin;

  // softmax state of rows 8nt + 2qi and 8nt + 2qi + 1 (HALVES: row qi) over this warp's tokens
  float m_run[NT][RPT], l_run[NT][RPT];
  float zsum[G::NVG][NT][RPT];             // sum_j p_j z_{j,g}, lane-partial
  float co[NT][8][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      m_run[nt][i] = -INFINITY;
      l_run[nt][i] = 0.0f;
#pragma unroll
      for (int g = 0; g < G::NVG; ++g) zsum[g][nt][i] = 0.0f;
    }
#pragma unroll
    for (int mv = 0; mv < 8; ++mv)
#pragma unroll
      for (int e = 0; e < 4; ++e) co[nt][mv][e] = 0.0f;
  }
  bool failed = false;
  const float alpha = a.score_scale;
  constexpr float kMid = static_cast<float>(1 << (VB - 1));   // centre of the value codes
  const float alpha24 = a.score_scale * 16777216.0f;          // undoes the 2^-24 of subnormal codes

  // Weights are 2^(score - reference + lift).  Their products with a value scale are rounded to fp16
  // below, so `lift` puts them where fp16 is exact to 2^-11: the largest scale so far, times 2^lift, lies
  // in [2^11, 2^15], whatever the values' magnitude (unlifted, values around 1e-4 came out with errors
  // of a percent: their products with most weights are subnormal).  A scale above 2^(15 - lift) moves
  // it; the smallest one there is, 2^-24, passes the initial 2^-49.  The fp16 list keeps 0: its weights
  // are rounded without a scale.  The check costs 0 to 3%.
  float lift = quant ? 64.0f : 0.0f;

  auto scale_row = [&](int nt, float f0, float f1) {
    l_run[nt][0] *= f0;
    if constexpr (!HALVES) l_run[nt][RPT - 1] *= f1;
#pragma unroll
    for (int g = 0; g < G::NVG; ++g) {
      zsum[g][nt][0] *= f0;
      if constexpr (!HALVES) zsum[g][nt][RPT - 1] *= f1;
    }
#pragma unroll
    for (int mv = 0; mv < 8; ++mv) {
      co[nt][mv][0] *= f0;
      co[nt][mv][1] *= HALVES ? f0 : f1;
      co[nt][mv][2] *= f0;
      co[nt][mv][3] *= HALVES ? f0 : f1;
    }
  };
  // Moves the references of an n-tile's rows to their maxima.  They do not lag behind: weights stay at
  // most 2^lift, and those products at most 2^15 (a lag of 8 measured 4% less time at most).
  auto rescale = [&](int nt, float g0, float g1) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      g0 = fmaxf(g0, __shfl_xor_sync(0xffffffffu, g0, o));
      if constexpr (!HALVES) g1 = fmaxf(g1, __shfl_xor_sync(0xffffffffu, g1, o));
    }
    const bool mv0 = g0 > m_run[nt][0], mv1 = !HALVES && g1 > m_run[nt][RPT - 1];
    if (__any_sync(0xffffffffu, mv0 || mv1)) {
      const float f0 = mv0 ? ptx::ex2(m_run[nt][0] - g0) : 1.0f, f1 = mv1 ? ptx::ex2(m_run[nt][RPT - 1] - g1) : 1.0f;
      if (mv0) m_run[nt][0] = g0;
      if (mv1) m_run[nt][RPT - 1] = g1;
      scale_row(nt, f0, f1);
    }
  };

  if (quant) {
    // B operands in shared memory: q, and q scaled by 2^-p per k-slot
    if (warp == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int s = 0; s < KSTEPS; ++s)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int omega = qi * G::WPT + s / G::KSPW;
            const int rho = 2 * (s % G::KSPW) + j;
            const int c_lo = G::CPW * omega + rho, c_hi = c_lo + 16 / KB;
            const __half2 pair = qok[nt] ? __halves2half2(qrow[nt][c_lo], qrow[nt][c_hi]) : __float2half2_rn(0.0f);
            const float f = 1.0f / static_cast<float>(1 << mma::key_reg_shift<KB>(rho));
            const int at = nt * 2 * KSTEPS * 32 + mma::qb_index(2 * s + j, lane);
            sm_qf[at] = ptx::h2_as_u32(__hmul2(pair, __float2half2_rn(f)));
            sm_qb[at] = ptx::h2_as_u32(pair);
          }
    }
    float* sm_qt = reinterpret_cast<float*>(smem + SM::kQt);
    if constexpr (SR > 0) {
      // U_h^T q of every row: each lane sums DK/32 channels, then the warp reduces
      const float* uh = cb.side_u + static_cast<size_t>(h) * DK * SR;
      for (int r = warp; r < 8 * NT; r += kWarps) {
        const bool ok = rb + r < n_rows && (rb + r) % a.T < sw.n;
        const __half* qw = a.q + (static_cast<size_t>(bh) * n_rows + (ok ? rb + r : 0)) * DK;
        float acc[SR];
#pragma unroll
        for (int i = 0; i < SR; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int cc = 0; cc < DK / 32; ++cc) {
          const int ch = lane + 32 * cc;
          const float qc = ok ? __half2float(qw[ch]) : 0.0f;
#pragma unroll
          for (int i4 = 0; i4 < SR; i4 += 4) {
            const float4 u4 = *reinterpret_cast<const float4*>(uh + ch * SR + i4);
            acc[i4] = fmaf(u4.x, qc, acc[i4]);
            acc[i4 + 1] = fmaf(u4.y, qc, acc[i4 + 1]);
            acc[i4 + 2] = fmaf(u4.z, qc, acc[i4 + 2]);
            acc[i4 + 3] = fmaf(u4.w, qc, acc[i4 + 3]);
          }
        }
#pragma unroll
        for (int i = 0; i < SR; ++i) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
          if (lane == 0) sm_qt[r * SR + i] = acc[i];
        }
      }
    }
    __syncthreads();
    // retained positions, one per lane (ascending), for masking the quantized tiles
    const int ret_pos = lane < sw.n_ret ? retained_position(sw.Q, lane) : -1;
    const mma::StageLayout L = mma::quant_stage_layout(GK, DK, KB, VB, G::NVG, Z::ZB, SR);
    constexpr int MT = GK / 16;
    const bool swap = qi >= 2;
    const uint32_t sel_lo = swap ? 0x1054u : 0x5410u;
    const uint32_t sel_hi = swap ? 0x3276u : 0x7632u;
    constexpr int RING = RG::RING_Q, STAGE = RG::STAGE_Q;
    int* sm_page = reinterpret_cast<int*>(smem + SM::kPage);
    auto table_entry = [&](int k) {
      const int gg = unit_begin + k;
      return cb.table + (b * d.max_groups + (KVQ_IN_BOUNDS(d, kSiteChunkTable, gg, d.max_groups) ? gg : 0));
    };
    auto group_of = [&](int k, bool fetched) -> size_t {
      if (!d.paged) return static_cast<size_t>(bh) * d.max_groups + unit_begin + k;
      int page;
      if (fetched) {
        ptx::cp_async_wait_all();
        page = sm_page[warp];
      } else {
        page = __ldg(table_entry(k));
      }
      return static_cast<size_t>(page) * d.Hkv + h;
    };
    // one lane copies unit k (a whole key group: 4 contiguous runs) into stage k % RING
    auto issue = [&](int k, size_t gi) {
      // (bounds-check builds) a group outside the buffers is replaced by group 0
      if (!KVQ_IN_BOUNDS(d, kSiteChunkGroup, static_cast<long long>(gi), quant_groups(d))) gi = 0;
      const int st = k % RING;
      const uint32_t bar = bar0 + 8 * st, dst = stages_s + st * STAGE;
      sm_issued[st] += 1;
      sm_tag[st] = k;
      ptx::mbar_arrive_expect_tx(bar, L.bytes);
      const size_t tok = gi * GK;
      ptx::bulk_g2s(dst + L.k_off, cb.kcode + tok * G::KW, GK * G::KBYTES_ROW, bar);
      ptx::bulk_g2s(dst + L.kmeta_off, cb.ksz + gi * DK, DK * 4, bar);
      ptx::bulk_g2s(dst + L.v_off, cb.vcode + tok * G::VW, GK * G::VBYTES_ROW, bar);
      ptx::bulk_g2s(dst + L.vmeta_off, cb.vsz + tok * G::NVG, GK * G::NVG * 4, bar);
      if constexpr (SR > 0) {
        ptx::bulk_g2s(dst + L.z_off, cb.zcode + tok * Z::ZB, GK * Z::ZB, bar);
        ptx::bulk_g2s(dst + L.zmeta_off, cb.zsz + gi * SR, SR * 4, bar);
      }
    };
    if (threadIdx.x == 0)
      for (int k = 0; k < RING && k < n_units; ++k) issue(k, group_of(k, false));

    for (int k = warp; k < n_units; k += kWarps) {
      // the page the stage is refilled with after this unit, fetched early
      if (d.paged && lane == 0 && k + RING < n_units)
        ptx::cp_async_4(ptx::smem_addr(sm_page + warp), table_entry(k + RING));
      const int st = k % RING;
      const bool ok = ptx::wait_equal_bounded(sm_tag + st, k, kWaitLimitNs) &&
                      ptx::mbar_wait_bounded(bar0 + 8 * st, (k / RING) & 1, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, ok)) {
        failed = true;
        break;
      }
      const unsigned char* S = stages + st * STAGE;
      const uint32_t* skc = reinterpret_cast<const uint32_t*>(S + L.k_off);
      const uint32_t* skm = reinterpret_cast<const uint32_t*>(S + L.kmeta_off);
      const uint32_t* svc = reinterpret_cast<const uint32_t*>(S + L.v_off);
      const uint32_t* svm = reinterpret_cast<const uint32_t*>(S + L.vmeta_off);

      // ---- the lift of the weights follows the group's value scales ----
      {
        constexpr int W = GK * G::NVG / 32;      // the lane's share of the (scale, zero) pairs
        uint32_t sz[W];
        mma::load_words<W>(svm + lane * W, sz);
        __half2 mx = ptx::u32_as_h2(sz[0]);
#pragma unroll
        for (int i = 1; i < W; ++i) mx = __hmax2(mx, ptx::u32_as_h2(sz[i]));
        float top = __low2float(mx);
        if (__any_sync(0xffffffffu, top > ptx::ex2(15.0f - lift))) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;      // 2^e <= top < 2^(e + 1)
          const float to = static_cast<float>(11 - e), f = ptx::ex2(to - lift);
          lift = to;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) scale_row(nt, f, f);
        }
      }
      // ---- group prologue: B = q * s, and the zero-point bias ----
      uint32_t bq[NT][KSTEPS][2];
      float cbias[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) cbias[nt][e] = 0.0f;
#pragma unroll
      for (int u = 0; u < G::WPT; ++u) {
        uint32_t meta[G::CPW];
#pragma unroll
        for (int c4 = 0; c4 < G::CPW; c4 += 4) {
          // word qi * WPT + u: its block is stored at position u * 4 + qi
          const uint4 v4 = *reinterpret_cast<const uint4*>(skm + G::CPW * (u * 4 + qi) + c4);
          meta[c4] = v4.x;
          meta[c4 + 1] = v4.y;
          meta[c4 + 2] = v4.z;
          meta[c4 + 3] = v4.w;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          constexpr int E = 2 * G::KSPW;
          uint32_t qbx[E], qfx[E];
          constexpr int W = E >= 4 ? 4 : E;
#pragma unroll
          for (int c4 = 0; c4 < E; c4 += W) {
            mma::load_words<W>(sm_qb + nt * 2 * KSTEPS * 32 + mma::qb_index(u * E + c4, lane), qbx + c4);
            mma::load_words<W>(sm_qf + nt * 2 * KSTEPS * 32 + mma::qb_index(u * E + c4, lane), qfx + c4);
          }
#pragma unroll
          for (int ls = 0; ls < G::KSPW; ++ls) {
            const int s = u * G::KSPW + ls;
            uint32_t za[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // the word's block holds (s_c, s_c+16/KB) for each register, then the zeros
              const int rho = 2 * ls + j;
              za[j] = meta[G::RPW + rho];
              const __half2 qs = ptx::u32_as_h2(qfx[2 * ls + j]), sc = ptx::u32_as_h2(meta[rho]), hi = __hmul2(qs, sc);
              bq[nt][s][j] = ptx::h2_as_u32(low ? __hfma2(qs, sc, __hneg2(hi)) : hi);
            }
            ptx::mma_16816(cbias[nt], za[0], za[0], za[1], za[1], qbx[2 * ls], qbx[2 * ls + 1]);
          }
        }
      }

      // the side code: its scales into U_h^T q, its zeros into the bias
      uint32_t bz[NT];
      if constexpr (SR > 0) {
        const __half2* zm = reinterpret_cast<const __half2*>(S + L.zmeta_off);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          bz[nt] = 0u;
          if (qi < Z::NQ) {
            const float f = 1.0f / static_cast<float>(1 << Z::pos(qi));
            const float* qt = sm_qt + (8 * nt + (HALVES ? qr >> 1 : qr)) * SR;
            const float x0 = qt[qi] * __low2float(zm[qi]) * f, x1 = qt[qi + Z::NQ] * __low2float(zm[qi + Z::NQ]) * f;
            const __half2 hi = __floats2half2_rn(x0, x1);
            bz[nt] = ptx::h2_as_u32(low ? __floats2half2_rn(x0 - __low2float(hi), x1 - __high2float(hi)) : hi);
          }
#pragma unroll
          for (int i = 0; i < SR; ++i) {
            const float zero = __high2float(zm[i]);
#pragma unroll
            for (int r = 0; r < RPT; ++r)
              cbias[nt][r] = fmaf(sm_qt[(8 * nt + RPT * qi + r) * SR + i], zero, cbias[nt][r]);
          }
        }
      }

      // ---- scores of the whole group: tokens 16 mt + qr, + 8; the thread's rows of every n-tile ----
      float sc[NT][MT][2 * RPT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float cs[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) cs[nt][e] = 0.0f;
        const int t0 = 16 * mt + qr;
        uint32_t w0[G::WPT], w1[G::WPT];
        mma::load_words<G::WPT>(skc + t0 * G::KW + qi * G::WPT, w0);
        mma::load_words<G::WPT>(skc + (t0 + 8) * G::KW + qi * G::WPT, w1);
#pragma unroll
        for (int u = 0; u < G::WPT; ++u) {
          uint32_t r0[G::RPW], r1[G::RPW];
          mma::unpack_key_word<KB>(w0[u], r0);
          mma::unpack_key_word<KB>(w1[u], r1);
#pragma unroll
          for (int ls = 0; ls < G::KSPW; ++ls) {
            const int s = u * G::KSPW + ls;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              ptx::mma_16816(cs[nt], r0[2 * ls], r1[2 * ls], r0[2 * ls + 1], r1[2 * ls + 1], bq[nt][s][0], bq[nt][s][1]);
          }
        }
        if constexpr (SR > 0) {
          const unsigned char* zr = S + L.z_off;
          uint32_t x0, x1;
          if constexpr (Z::ZB == 4) {
            x0 = *reinterpret_cast<const uint32_t*>(zr + t0 * 4);
            x1 = *reinterpret_cast<const uint32_t*>(zr + (t0 + 8) * 4);
          } else {
            // (c0 c1 | c2 c3) of a 16-bit row -> c0 c1 in the low half, c2 c3 in the high half
            x0 = ptx::prmt(*reinterpret_cast<const uint16_t*>(zr + t0 * 2), 0u, 0x0100u);
            x1 = ptx::prmt(*reinterpret_cast<const uint16_t*>(zr + (t0 + 8) * 2), 0u, 0x0100u);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            ptx::mma_1688(cs[nt], (x0 >> Z::shift(qi)) & Z::mask(qi), (x1 >> Z::shift(qi)) & Z::mask(qi), bz[nt]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2 * RPT; ++e)
            sc[nt][mt][e] = fmaf(HALVES ? cs[nt][2 * e] + cs[nt][2 * e + 1] : cs[nt][e], alpha24, cbias[nt][e % RPT] * alpha);
      }
      // retained tokens of this group are read from the fp16 list: mask them here
      const int g0 = (unit_begin + k) * GK;
      unsigned hits = __ballot_sync(0xffffffffu, ret_pos >= g0 && ret_pos < g0 + GK);
      while (hits) {
        const int src = __ffs(hits) - 1;
        hits &= hits - 1;
        const int off = __shfl_sync(0xffffffffu, ret_pos, src) - g0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2 * RPT; ++e)
              if (off == 16 * mt + qr + (e / RPT) * 8) sc[nt][mt][e] = -INFINITY;
          }
      }
      // ---- online softmax update for the group ----
      float m_use[NT][RPT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          x0 = fmaxf(x0, fmaxf(sc[nt][mt][0], sc[nt][mt][RPT]));
          x1 = fmaxf(x1, fmaxf(sc[nt][mt][RPT - 1], sc[nt][mt][2 * RPT - 1]));
        }
        rescale(nt, x0, x1);
#pragma unroll
        for (int i = 0; i < RPT; ++i) m_use[nt][i] = (m_run[nt][i] == -INFINITY ? 0.0f : m_run[nt][i]) - lift;
      }

      // ---- p.V over the group ----
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int t0 = 16 * mt + qr;
        float p[NT][2 * RPT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2 * RPT; ++e) p[nt][e] = ptx::ex2(sc[nt][mt][e] - m_use[nt][e % RPT]);
#pragma unroll
          for (int i = 0; i < RPT; ++i) l_run[nt][i] += p[nt][i] + p[nt][RPT + i];
        }
        // value (scale, zero) of the two tokens this thread weights
        uint32_t vm0[G::NVG], vm1[G::NVG];
        mma::load_words<G::NVG>(svm + t0 * G::NVG, vm0);
        mma::load_words<G::NVG>(svm + (t0 + 8) * G::NVG, vm1);
        // value words: tokens 2qi, 2qi+1, 2qi+8, 2qi+9 of the tile, swapped for qi >= 2
        const int ta = 16 * mt + 2 * qi + (swap ? 1 : 0);
        const int tb = 16 * mt + 2 * qi + (swap ? 0 : 1);
        // 16-bit runs (a value group's row is 16 bytes) come through ldmatrix.trans
        constexpr bool kLdm = G::RUN == 16 && GV * VB / 8 == 16 && G::NVG % 2 == 0;
        uint32_t xv[G::NVG][2];
        if constexpr (kLdm) {
          const int j = lane >> 3, r = lane & 7;
#pragma unroll
          for (int g4 = 0; g4 < G::NVG; g4 += 2)
            ptx::ldmatrix_x4_trans(ptx::smem_addr(svc) + (16 * mt + 8 * (j & 1) + r) * G::VBYTES_ROW + (g4 + (j >> 1)) * 16,
                                   xv[g4][0], xv[g4][1], xv[g4 + 1][0], xv[g4 + 1][1]);
        }
#pragma unroll
        for (int gg = 0; gg < G::NVG; ++gg) {
          const float2 f0 = __half22float2(ptx::u32_as_h2(vm0[gg]));
          const float2 f1 = __half22float2(ptx::u32_as_h2(vm1[gg]));
          // with centred codes (c - mid) the zero-point sum takes z + mid * s instead of z
          const float zc0 = fmaf(kMid, f0.x, f0.y), zc1 = fmaf(kMid, f1.x, f1.y);
          uint32_t bp[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < RPT; ++i)
              zsum[gg][nt][i] = fmaf(p[nt][i], zc0, fmaf(p[nt][RPT + i], zc1, zsum[gg][nt][i]));
            bp[nt][0] = ptx::movmatrix_trans(weights<HALVES>(p[nt][0] * f0.x, p[nt][RPT - 1] * f0.x));
            bp[nt][1] = ptx::movmatrix_trans(weights<HALVES>(p[nt][RPT] * f1.x, p[nt][2 * RPT - 1] * f1.x));
          }
          const int bit0 = (gg * GV + qr * G::CPG) * VB;
          const int wv = bit0 >> 5, ob = bit0 & 31;
          uint32_t ra[G::CPG], rb[G::CPG];   // codes of tokens (2qi, 2qi+1) and (2qi+8, 2qi+9)
          if constexpr (kLdm) {
            mma::unpack_value_piece16<VB>(xv[gg][0], ra);
            mma::unpack_value_piece16<VB>(xv[gg][1], rb);
          } else {
            const uint32_t wa0 = svc[ta * G::VW + wv], wb0 = svc[tb * G::VW + wv];
            const uint32_t wa1 = svc[(ta + 8) * G::VW + wv], wb1 = svc[(tb + 8) * G::VW + wv];
            if constexpr (G::RUN == 8) {
              const uint32_t bsel = static_cast<uint32_t>(ob >> 3);
              const uint32_t s8 = swap ? ((4 + bsel) | ((4 + bsel) << 4) | (bsel << 8) | (bsel << 12))
                                       : (bsel | (bsel << 4) | ((4 + bsel) << 8) | ((4 + bsel) << 12));
              mma::unpack_value_piece8<VB>(ptx::prmt(wa0, wb0, s8), ra);
              mma::unpack_value_piece8<VB>(ptx::prmt(wa1, wb1, s8), rb);
            } else if constexpr (G::RUN == 16) {
              const uint32_t s16 = ob ? sel_hi : sel_lo;
              mma::unpack_value_piece16<VB>(ptx::prmt(wa0, wb0, s16), ra);
              mma::unpack_value_piece16<VB>(ptx::prmt(wa1, wb1, s16), rb);
            } else {
              constexpr int n16 = 16 / VB;
              mma::unpack_value_piece16<VB>(ptx::prmt(wa0, wb0, sel_lo), ra);
              mma::unpack_value_piece16<VB>(ptx::prmt(wa0, wb0, sel_hi), ra + n16);
              mma::unpack_value_piece16<VB>(ptx::prmt(wa1, wb1, sel_lo), rb);
              mma::unpack_value_piece16<VB>(ptx::prmt(wa1, wb1, sel_hi), rb + n16);
            }
          }
          // centred codes (c - mid) * 2^(p-24): an exact fp16 subnormal subtraction
#pragma unroll
          for (int e = 0; e < G::CPG; ++e) {
            const uint32_t mid = (1u << (VB - 1 + mma::value_code_shift<VB, G::RUN>(e))) * 0x00010001u;
            ra[e] = ptx::h2_as_u32(__hsub2(ptx::u32_as_h2(ra[e]), ptx::u32_as_h2(mid)));
            rb[e] = ptx::h2_as_u32(__hsub2(ptx::u32_as_h2(rb[e]), ptx::u32_as_h2(mid)));
          }
#pragma unroll
          for (int ml = 0; ml < G::MPG; ++ml)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              ptx::mma_16816(co[nt][gg * G::MPG + ml], ra[ml], ra[ml + G::MPG], rb[ml], rb[ml + G::MPG], bp[nt][0], bp[nt][1]);
        }
      }
      // ---- release the stage: refill it with unit k + RING ----
      __syncwarp();
      if (lane == 0 && k + RING < n_units) {
        ptx::fence_proxy_async_smem();
        issue(k + RING, group_of(k + RING, true));
      }
    }
  } else {
    // ---------------- fp16 rows: retained tokens, the window, the new tokens ----------------
    constexpr int RING = RG::RING_F, STAGE = RG::STAGE_F;
    uint32_t qn[NT][KSTEPS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < KSTEPS; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = 16 * s + 2 * qi + 8 * j;
          qn[nt][s][j] = qok[nt] && !low ? ptx::h2_as_u32(__halves2half2(qrow[nt][c], qrow[nt][c + 1])) : 0u;
        }
    // stale shared memory must hold finite values: masked rows multiply p = 0
    for (int i = threadIdx.x; i < RING * STAGE / 16; i += kThreads)
      reinterpret_cast<uint4*>(stages)[i] = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
    __syncthreads();
    // the 32 lanes of one warp copy the up to 16 key and 16 value rows of unit k
    auto issue = [&](int k) {
      const int st = k % RING;
      const uint32_t bar = bar0 + 8 * st, dst = stages_s + st * STAGE;
      const int e0 = list_begin + 16 * k, nvalid = min(16, list_end - e0);
      if (lane == 0) {
        sm_issued[st] += 1;
        sm_tag[st] = k;
        ptx::mbar_arrive_expect_tx(bar, nvalid * (DK + kDV) * 2);
      }
      __syncwarp();
      const int row = lane & 15;
      if (row < nvalid) {
        const int e = e0 + row;
        long long slot;
        const __half *bk, *bv;
        if (e >= n_old) {
          slot = static_cast<long long>(bh) * a.T + (e - n_old);
          bk = a.k_new;
          bv = a.v_new;
        } else if (e < sw.n_ret) {
          slot = static_cast<long long>(bh) * kMaxRetained + e;
          if (!KVQ_IN_BOUNDS(d, kSiteChunkFp16, slot, ret_rows(d))) slot = 0;
          bk = cb.ret_k;
          bv = cb.ret_v;
        } else {
          slot = static_cast<long long>(bh) * d.cap + (sw.Q + e - sw.n_ret) % d.cap;
          if (!KVQ_IN_BOUNDS(d, kSiteChunkFp16, slot, win_rows(d))) slot = 0;
          bk = cb.win_k;
          bv = cb.win_v;
        }
        if (lane < 16)
          ptx::bulk_g2s(dst + row * R::KST, bk + slot * DK, DK * 2, bar);
        else
          ptx::bulk_g2s(dst + 16 * R::KST + row * R::VST, bv + slot * kDV, kDV * 2, bar);
      }
    };
    const int mask_words = (a.T + 31) / 32;
    // whether query row r sees entry e of the list
    auto sees = [&](int e, int r) {
      if (e >= list_end) return false;
      if (e < n_old) return true;
      const int j = e - n_old, t = r % a.T;
      if (r >= n_rows || t >= sw.n) return false;
      return a.mask ? (a.mask[(static_cast<long long>(b) * a.T + t) * mask_words + j / 32] >> (j & 31) & 1u) != 0 : j <= t;
    };
    if (warp == 0)
      for (int k = 0; k < RING && k < n_units; ++k) issue(k);
    for (int k = warp; k < n_units; k += kWarps) {
      const int st = k % RING;
      const bool ok = ptx::wait_equal_bounded(sm_tag + st, k, kWaitLimitNs) &&
                      ptx::mbar_wait_bounded(bar0 + 8 * st, (k / RING) & 1, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, ok)) {
        failed = true;
        break;
      }
      const uint32_t S = stages_s + st * STAGE;
      const int e0 = list_begin + 16 * k;
      float cs[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[nt][e] = 0.0f;
      const int mi = lane >> 3;                         // which 8x8 matrix this lane addresses
      const int arow = (mi & 1) * 8 + (lane & 7);
#pragma unroll
      for (int s = 0; s < KSTEPS; ++s) {
        uint32_t a0, a1, a2, a3;
        ptx::ldmatrix_x4(S + arow * R::KST + (16 * s + (mi >> 1) * 8) * 2, a0, a1, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ptx::mma_16816(cs[nt], a0, a1, a2, a3, qn[nt][s][0], qn[nt][s][1]);
      }
      uint32_t bp[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2 * RPT; ++e) {
          // (HALVES: the queries stand in the high columns alone)
          const float x = cs[nt][HALVES ? 2 * e : e];
          cs[nt][e] = sees(e0 + qr + 8 * (e / RPT), rb + 8 * nt + RPT * qi + e % RPT) ? x * alpha : -INFINITY;
        }
        rescale(nt, fmaxf(cs[nt][0], cs[nt][RPT]), fmaxf(cs[nt][RPT - 1], cs[nt][2 * RPT - 1]));
        float p[2 * RPT];
#pragma unroll
        for (int e = 0; e < 2 * RPT; ++e) {
          const float m = m_run[nt][e % RPT];
          p[e] = ptx::ex2(cs[nt][e] - (m == -INFINITY ? 0.0f : m));
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) l_run[nt][i] += p[i] + p[RPT + i];
        bp[nt][0] = ptx::movmatrix_trans(weights<HALVES>(p[0], p[RPT - 1]));
        bp[nt][1] = ptx::movmatrix_trans(weights<HALVES>(p[RPT], p[2 * RPT - 1]));
      }
      // p.V: A = V^T tiles via ldmatrix.trans (rows = tokens in shared memory)
      const int vrow = (mi >> 1) * 8 + (lane & 7);
#pragma unroll
      for (int mv = 0; mv < 8; ++mv) {
        uint32_t a0, a1, a2, a3;
        ptx::ldmatrix_x4_trans(S + 16 * R::KST + vrow * R::VST + (16 * mv + (mi & 1) * 8) * 2, a0, a1, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ptx::mma_16816(co[nt][mv], a0, a1, a2, a3, bp[nt][0], bp[nt][1]);
      }
      __syncwarp();
      if (k + RING < n_units) {
        if (lane == 0) ptx::fence_proxy_async_smem();
        issue(k + RING);
      }
    }
  }

  // A bounded wait gave up: flag it, then wait (bounded) for the last copy issued into every stage
  // so that no copy lands in shared memory after the CTA has exited.
  if (failed && lane == 0) {
    atomicOr(a.status, KVQ_STATUS_TIMEOUT);
    atomicOr(sm_fail, 1);
  }
  if (d.paged) ptx::cp_async_wait_all();          // a page fetch of a unit given up on
  __syncthreads();
  if (*sm_fail) {
    if (threadIdx.x < ring && sm_issued[threadIdx.x] > 0)
      ptx::mbar_wait_bounded(bar0 + 8 * threadIdx.x, (sm_issued[threadIdx.x] - 1) & 1, kWaitLimitNs);
    failed = true;     // the CTA's partial is dropped as a whole
  }

  // ---------------- warp totals, then the CTA merge ----------------
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l_run[nt][i] += __shfl_xor_sync(0xffffffffu, l_run[nt][i], o);
#pragma unroll
        for (int gg = 0; gg < G::NVG; ++gg) zsum[gg][nt][i] += __shfl_xor_sync(0xffffffffu, zsum[gg][nt][i], o);
      }
      if (failed) {
        m_run[nt][i] = -INFINITY;
        l_run[nt][i] = 0.0f;
      }
    }
  __syncthreads();   // every warp is done with the stages: reuse them for the merge
  constexpr int NR = ROWS;
  float* sm_o = reinterpret_cast<float*>(smem + SM::kStages);        // [kWarps][NR][kDV]
  float* sm_ml = sm_o + kWarps * NR * kDV;                           // [kWarps][NR][2]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = 8 * nt + RPT * qi + i;
      float* dst = sm_o + (warp * NR + r) * kDV;
#pragma unroll
      for (int mv = 0; mv < 8; ++mv) {
        float o0 = co[nt][mv][i], o1 = co[nt][mv][2 + i];
        if constexpr (HALVES) {
          o0 += co[nt][mv][1];
          o1 += co[nt][mv][3];
        }
        int c0, c1;
        if (quant) {
          const int gg = mv / G::MPG, ml = mv % G::MPG;
          c0 = gg * GV + qr * G::CPG + ml;
          c1 = c0 + G::MPG;
          o0 = fmaf(o0, static_cast<float>(1 << (24 - mma::value_code_shift<VB, G::RUN>(ml))), zsum[gg][nt][i]);
          o1 = fmaf(o1, static_cast<float>(1 << (24 - mma::value_code_shift<VB, G::RUN>(ml + G::MPG))), zsum[gg][nt][i]);
        } else {
          c0 = 16 * mv + qr;
          c1 = c0 + 8;
        }
        dst[c0] = failed ? 0.0f : o0;
        dst[c1] = failed ? 0.0f : o1;
      }
      if (qr == 0) {
        sm_ml[(warp * NR + r) * 2] = m_run[nt][i] - lift;      // -inf stays -inf
        sm_ml[(warp * NR + r) * 2 + 1] = l_run[nt][i];
      }
    }
  __syncthreads();
  for (int idx = threadIdx.x; idx < min(NR, n_rows - rb) * kDV; idx += kThreads) {
    const int r = idx / kDV, c = idx % kDV;
    if ((rb + r) % a.T >= sw.n) continue;
    float M = -INFINITY;
#pragma unroll
    for (int ww = 0; ww < kWarps; ++ww) M = fmaxf(M, sm_ml[(ww * NR + r) * 2]);
    float acc = 0.0f, lsum = 0.0f;
#pragma unroll
    for (int ww = 0; ww < kWarps; ++ww) {
      const float mw = sm_ml[(ww * NR + r) * 2];
      const float wt = (mw == -INFINITY) ? 0.0f : exp2f(mw - M);
      acc = fmaf(wt, sm_o[(ww * NR + r) * kDV + c], acc);
      lsum = fmaf(wt, sm_ml[(ww * NR + r) * 2 + 1], lsum);
    }
    const long long row = static_cast<long long>(bh) * n_rows + rb + r, pi = row * a.splits + split;
    if (!KVQ_IN_BOUNDS(d, kSiteChunkPartial, row, static_cast<long long>(d.B) * d.Hq * a.T)) continue;
    if (a.splits == 1) {
      a.out[row * kDV + c] = __float2half_rn(lsum > 0.0f ? acc / lsum : 0.0f);
    } else {
      a.o[pi * kDV + c] = acc;
      if (c == 0) a.ml[pi] = make_float2(M, lsum);
    }
  }
}

template <int KB, int VB, int DK, int GV, int GK, int SR, int SQ, int ROWS>
cudaError_t launch(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  using RG = Rings<KB, VB, DK, GV, GK, SR, SQ, ROWS>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(chunk_few_kernel<KB, VB, DK, GV, GK, SR, SQ, ROWS>, RG::BYTES);
  if (e != cudaSuccess) return e;
  const int blocks = (d.n_rep * a.T + ROWS - 1) / ROWS;
  chunk_few_kernel<KB, VB, DK, GV, GK, SR, SQ, ROWS><<<dim3(a.splits * blocks, d.Hkv, d.B), kThreads, RG::BYTES, s>>>(d, c, a);
  return cudaGetLastError();
}

// The built instances, F(KB, VB, DK, GV, GK, SR, SQ): the decode kernel's bit widths, group sizes and
// side codes.
#define KVQ_CHUNK_FEW_4(F)                                                                     \
  F(4, 2, 128, 64, 64, 0, 4) F(4, 2, 128, 32, 32, 0, 4) F(4, 2, 32, 32, 32, 0, 4)              \
  F(4, 2, 32, 64, 64, 0, 4) F(4, 4, 128, 64, 64, 0, 4) F(4, 4, 32, 64, 64, 0, 4)
#define KVQ_CHUNK_FEW_28(F)                                                                    \
  F(8, 4, 128, 64, 64, 0, 4) F(8, 4, 128, 32, 32, 0, 4) F(8, 4, 32, 64, 64, 0, 4)              \
  F(2, 2, 128, 64, 64, 0, 4) F(2, 2, 128, 32, 32, 0, 4)
#define KVQ_CHUNK_FEW_SIDE(F)                                                                  \
  F(4, 2, 128, 64, 64, 4, 4) F(4, 2, 128, 64, 64, 4, 8) F(4, 2, 128, 64, 64, 8, 4)             \
  F(2, 2, 128, 64, 64, 4, 4) F(2, 2, 128, 64, 64, 4, 8) F(2, 2, 128, 64, 64, 8, 4)

using LaunchFn = cudaError_t (*)(const Dims&, const CacheBufs&, const ChunkArgs&, cudaStream_t);
// The instance for a cache and number of rows, or null (each file knows its own).
LaunchFn find_4(const Dims& d, int rows);
LaunchFn find_28(const Dims& d, int rows);
LaunchFn find_side(const Dims& d, int rows);

#define KVQ_CHUNK_FEW_ENTRY(KB, VB, DK, GV, GK, SR, SQ)                                        \
  if (d.kb == KB && d.vb == VB && d.dk == DK && d.gv == GV && d.gk == GK && d.sr == SR &&      \
      (SR == 0 || d.sq == SQ))                                                                 \
    return chunk_few_block(d, rows) == 4    ? &launch<KB, VB, DK, GV, GK, SR, SQ, 4>              \
           : chunk_few_block(d, rows) == 8  ? &launch<KB, VB, DK, GV, GK, SR, SQ, 8>              \
           : chunk_few_block(d, rows) == 16 ? &launch<KB, VB, DK, GV, GK, SR, SQ, 16>             \
                                            : &launch<KB, VB, DK, GV, GK, SR, SQ, 24>;

}  // namespace few
}  // namespace kvq
