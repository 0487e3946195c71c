// Chunk attention on the tensor cores (tcgen05, sm_100a), few query rows: up to 32 rows of a kv
// head over a packed cache and the new tokens.
//
// The tokens take the MMA's 128 rows and the queries its N columns, so a tile costs what its
// queries ask for instead of a 128-row tile of mostly padding:
//
//   S^T = K Q^T      A = the decoded keys, B = the queries (both K-major in shared memory);
//   O^T += V^T P^T   A = the decoded values (MN-major: no transposition), B = the weights, written
//                    to shared memory by the softmax threads, a token per 128-byte row.
//
// Roles: 8 producer warps decode token tiles (see chunk_tile.cuh), one warp copies packed tiles, one
// issues the MMAs (the scores of the next tile before the product of this one); four softmax warps
// own a token (a TMEM lane) per thread and all its N scores.  A row's maximum runs over threads, so
// it is not taken at all in the common case: the weights are formed with the reference of the
// tiles before, and only when a score passes it by more than 8 (a vote over the four warps) is the
// maximum found and O^T rescaled.  Row sums stay per thread and are reduced once at the end.
//
// Roundings as in chunk_wide.cu: decoded keys, values and weights to fp16 once each; the rest is
// fp32.  Bound: the decoding (about 16 instructions per 8 channels and 512 shared-memory
// wavefronts a tile) ahead of memory; MMA and softmax are small.
#include <algorithm>

#include "chunk_tile.cuh"

namespace kvq {
namespace {

using namespace chunk;

constexpr int kSoftmaxThreads = 128;
constexpr float kNone = -1e30f;               // the reference of a row that has seen no token
constexpr float kOver = kLazy + kBias;        // (references are kept with kBias taken off)

template <int DK, int N>
struct Layout {
  static constexpr int kThreads = kSoftmaxThreads + kProducers + 64;   // and a warp that copies, one that issues the MMAs
  static constexpr int KH = DK > 64 ? DK / 64 : 1;
  static constexpr int kK = 0;
  static constexpr int kV = kK + 2 * KH * kHalf;
  static constexpr int kP = kV + 2 * 2 * kHalf;
  static constexpr int kQ = kP + kHalf;
  static constexpr int kBars = kQ + KH * N * 128;
  static constexpr int kPages = kBars + 192;
  static constexpr int kRow = kPages + 64;                // per row: reference, factor, token; maxima or sums of the warps
  static constexpr int kRing = kRow + 7 * N * 4;
  static constexpr int kFixed = kRing + 1024;             // the base is aligned to 1024 by hand
  static_assert(kRing % 16 == 0, "bulk copies");
  static constexpr int kTmem = N == 16 ? 64 : 128;
};

enum Bars { kSFull = kTokenBars, kPFull = kSFull + 2, kPvDone, kDone };

template <int N>
__device__ __forceinline__ void tmem_ld_row(uint32_t addr, uint32_t (&x)[N]) {
  if constexpr (N == 32) {
    tmem_ld32(addr, x);
  } else {
    tmem_ld16(addr, x);
  }
  tmem_wait_ld();
}
// Whether any of the four softmax warps says so.
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 3, 128;" ::: "memory"); }

// Maxima over the warp's 32 tokens of N columns to out[0 .. N): each exchange halves the columns a
// lane is responsible for, 31 exchanges for 32 columns.
template <int N>
__device__ __forceinline__ void column_max(const uint32_t (&x)[N], float* out, int lane) {
#pragma unroll
  for (int c = 0; c < N; c += 16) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(x[c + i]);
#pragma unroll
    for (int h = 8; h > 0; h >>= 1) {
      const bool up = lane & h;               // the lane keeps the upper half of its columns
#pragma unroll
      for (int i = 0; i < h; ++i) {
        const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + h], h);
        v[i] = fmaxf(up ? v[i + h] : v[i], other);
      }
    }
    const float m = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
    if (lane < 16) out[c + lane] = m;
  }
}

template <int DK, int N>
__global__ void __launch_bounds__(Layout<DK, N>::kThreads, 1)
chunk_narrow_kernel(const __grid_constant__ Dims d, const __grid_constant__ CacheBufs cb,
                    const __grid_constant__ ChunkArgs a, int stages) {
  using Lay = Layout<DK, N>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  __shared__ uint32_t sm_tmem;
  __shared__ int sm_fail;

  const int split = blockIdx.x % a.splits, r0 = blockIdx.x / a.splits * N, h = blockIdx.y, b = blockIdx.z;
  const int bh = b * d.Hkv + h;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const SeqNew s = seq_new(a.seq, b, d.log_retain);
  const int n_rows = d.n_rep * a.T;
  Tiles t;
  if (!block_tiles(a, s, r0, min(r0 + N, n_rows) - 1, split, t)) return;
  const int n = t.end - t.begin;

  float* sm_m = reinterpret_cast<float*>(smem + Lay::kRow);     // [N] reference maxima - kBias
  float* sm_f = sm_m + N;                                       // [N] factors of the last rescale
  int* sm_t = reinterpret_cast<int*>(sm_f + N);                 // [N] token of the row (-1: no row)
  float* sm_w = reinterpret_cast<float*>(sm_t + N);             // [4][N] per warp: maxima, in the end sums
  const uint32_t bars = base + Lay::kBars;
  if (tid == 0) {
    init_token_bars(bars, kProducers / 32, kProducers / 32, 1);
    for (int i = 0; i < 2; ++i) ptx::mbar_init(bars + 8 * (kSFull + i), 1);
    ptx::mbar_init(bars + 8 * kPFull, kSoftmaxThreads / 32);
    ptx::mbar_init(bars + 8 * kPvDone, 1);
    ptx::mbar_init(bars + 8 * kDone, 1);
    ptx::fence_barrier_init();
    sm_fail = 0;
  }
  if (tid < N) {
    const int r = r0 + tid, tr = r % a.T;
    sm_m[tid] = kNone;
    sm_t[tid] = r < n_rows && tr < s.n ? tr : -1;
  }
  clear_ring(d, base + Lay::kRing, stages, tid, Lay::kThreads);
  if (warp == 0) tmem_alloc(ptx::smem_addr(&sm_tmem), Lay::kTmem);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm_tmem;
  const Waiter wait{&sm_fail};
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t to = tmem + 2 * N + lanes;

  constexpr int kCopyWarp = (kSoftmaxThreads + kProducers) / 32, kMmaWarp = kCopyWarp + 1;
  if (warp == kCopyWarp) {
    const Ctx c{d, cb, a, s, b, h, bh, __ffs(d.gk) - 1, __ffs(d.gv) - 1, __ffs(d.nvg) - 1,
                base + Lay::kRing, base + Lay::kPages, stages};
    with_bits(d, [&](auto kb, auto vb) {
      if constexpr (kb.value != 16) copy_tiles<kb.value, vb.value, DK>(c, t, lane, bars, wait);
    });
    __syncthreads();
  } else if (warp == kMmaWarp) {
    // S^T of tile u into TMEM columns (u & 1) N, once its keys are there
    auto score = [&](int u) -> bool {
      const int st = u & 1;
      if (!__all_sync(0xffffffffu, wait(bars + 8 * (kKFull + st), (u >> 1) & 1))) return false;
      fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < DK / 16; ++k)
          mma_ss(tmem + st * N, desc_sw128(base + Lay::kK + st * Lay::KH * kHalf + (k >> 2) * kHalf + (k & 3) * 32, 16),
                 desc_sw128(base + Lay::kQ + (k >> 2) * (N * 128) + (k & 3) * 32, 16), instr_desc(N, false, false), k > 0);
        commit(bars + 8 * (kSFull + st));
        commit(bars + 8 * (kKEmpty + st));
      }
      __syncwarp();
      return true;
    };
    bool live = n > 0 && score(0);
    for (int u = 0; live && u < n; ++u) {
      const int st = u & 1;
      // the other score buffer is free: its weights (tile u - 1) were waited for
      if (u + 1 < n && !score(u + 1)) break;
      live = __all_sync(0xffffffffu, wait(bars + 8 * kPFull, u & 1) && wait(bars + 8 * (kVFull + st), (u >> 1) & 1));
      if (!live) break;
      fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ss(tmem + 2 * N, desc_sw128(base + Lay::kV + st * 2 * kHalf + k * 2048, kHalf),
                 desc_sw128(base + Lay::kP + k * 2048, kHalf), instr_desc(N, true, true), u > 0 || k > 0);
        commit(bars + 8 * kPvDone);
        commit(bars + 8 * (kVEmpty + st));
      }
      __syncwarp();
    }
    // everything issued has to end before the CTA frees its TMEM, also after a wait that ran out
    if (elect_one()) commit(bars + 8 * kDone);
    __syncwarp();
    if (!ptx::mbar_wait_bounded(bars + 8 * kDone, 0, kWaitNs)) *wait.fail = 1;
    __syncthreads();
  } else if (tid >= kSoftmaxThreads) {
    const Ctx c{d, cb, a, s, b, h, bh, __ffs(d.gk) - 1, __ffs(d.gv) - 1, __ffs(d.nvg) - 1,
                base + Lay::kRing, base + Lay::kPages, stages};
    const int pt = tid - kSoftmaxThreads;
    with_bits(d, [&](auto kb, auto vb) {
      copy_queries<kb.value, DK, N>(c, r0, n_rows, pt, base + Lay::kQ);
      produce<kb.value, vb.value, DK, false>(c, t, pt, base + Lay::kK, base + Lay::kV, bars, wait);
    });
    __syncthreads();
  } else {
    float l[N];                               // the thread's share of the row sums
#pragma unroll
    for (int r = 0; r < N; ++r) l[r] = 0.0f;
    const float alpha = a.score_scale;
    const int mask_words = (a.T + 31) / 32;
    bool live = true;
    for (int u = 0; u < n; ++u) {
      // A wait that runs out ends the work, not the loop: the barriers count every warp.
      const int st = u & 1, ph = (u >> 1) & 1;
      live = live && __all_sync(0xffffffffu, wait(bars + 8 * (kSFull + st), ph));
      fence_after();
      // which rows see this thread's token
      const int tile = t.begin + u;
      const int kind = tile < t.nq ? 0 : tile < t.nq + t.nf ? 1 : 2;
      const int j = (tile - (kind > 0 ? t.nq : 0) - (kind > 1 ? t.nf : 0)) * kTile + tid;
      const bool there = kind == 0 ? j < s.Q && !(s.n_ret && is_retained(s.Q, j)) : j < (kind == 1 ? t.n_fp16 : t.n_vis);
      // the scores in log2 units, -inf where the row does not see the token
      uint32_t x[N];
      tmem_ld_row<N>(tmem + st * N + lanes, x);
      if (kind == 2) {
#pragma unroll
        for (int r = 0; r < N; ++r) {
          const int tr = sm_t[r];
          bool see = there && tr >= j;
          if (a.mask)
            see = there && tr >= 0 &&
                  (a.mask[(static_cast<long long>(b) * a.T + tr) * mask_words + j / 32] >> (j & 31) & 1u);
          x[r] = see ? __float_as_uint(__uint_as_float(x[r]) * alpha) : 0xff800000u;
        }
      } else {
#pragma unroll
        for (int r = 0; r < N; ++r) x[r] = there ? __float_as_uint(__uint_as_float(x[r]) * alpha) : 0xff800000u;
      }
      bool over = false;
#pragma unroll
      for (int r = 0; r < N; r += 4) {
        const float4 m = *reinterpret_cast<const float4*>(sm_m + r);
        over |= __uint_as_float(x[r]) > m.x + kOver || __uint_as_float(x[r + 1]) > m.y + kOver ||
                __uint_as_float(x[r + 2]) > m.z + kOver || __uint_as_float(x[r + 3]) > m.w + kOver;
      }
      const bool move = softmax_any(over);
      // P V of the tile before: done with the weights' buffer, and O^T is complete
      if (u > 0) live = live && __all_sync(0xffffffffu, wait(bars + 8 * kPvDone, (u - 1) & 1));
      if (move) {
        column_max<N>(x, sm_w + warp * N, lane);
        softmax_sync();
        if (tid < N) {
          const float m = sm_m[tid];
          const float m2 = fmaxf(m, fmaxf(fmaxf(sm_w[tid], sm_w[N + tid]), fmaxf(sm_w[2 * N + tid], sm_w[3 * N + tid])) - kBias);
          sm_f[tid] = ptx::ex2(m - m2);
          sm_m[tid] = m2;
        }
        softmax_sync();
        if (u > 0) {
          fence_after();
#pragma unroll
          for (int c0 = 0; c0 < N; c0 += 16) {
            uint32_t o[16];
            tmem_ld_row<16>(to + c0, o);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              l[c0 + r] *= sm_f[c0 + r];
              o[r] = __float_as_uint(__uint_as_float(o[r]) * sm_f[c0 + r]);
            }
            tmem_st16(to + c0, o);
          }
          tmem_wait_st();
        }
      }
      // the weights, eight rows a 16-byte chunk of the token's row
      const uint32_t prow = base + Lay::kP + tid * 128;
      uint32_t p[N / 2];
#pragma unroll
      for (int r = 0; r < N; r += 4) {
        const float4 m = *reinterpret_cast<const float4*>(sm_m + r);
        const float w0 = ptx::ex2(__uint_as_float(x[r]) - m.x), w1 = ptx::ex2(__uint_as_float(x[r + 1]) - m.y);
        const float w2 = ptx::ex2(__uint_as_float(x[r + 2]) - m.z), w3 = ptx::ex2(__uint_as_float(x[r + 3]) - m.w);
        l[r] += w0;
        l[r + 1] += w1;
        l[r + 2] += w2;
        l[r + 3] += w3;
        p[r / 2] = ptx::h2_as_u32(__floats2half2_rn(w0, w1));
        p[r / 2 + 1] = ptx::h2_as_u32(__floats2half2_rn(w2, w3));
      }
#pragma unroll
      for (int r = 0; r < N; r += 8)
        st_shared(prow + (((r >> 3) ^ (tid & 7)) << 4), make_uint4(p[r / 2], p[r / 2 + 1], p[r / 2 + 2], p[r / 2 + 3]));
      ptx::fence_proxy_async_smem();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * kPFull);
    }
    // ---------------- outputs ----------------
#pragma unroll
    for (int r = 0; r < N; ++r) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
      if (lane == (r & 31)) sm_w[warp * N + r] = l[r];
    }
    __syncthreads();          // all roles are done, the MMAs among them
    fence_after();
    if (sm_fail) {
      if (tid == 0) atomicOr(a.status, KVQ_STATUS_TIMEOUT);
    } else {
      // the thread's position among the value channels, in the order of VB-bit codes
      const int per = d.vb == 16 ? 1 : 32 / d.vb, q = tid & (per - 1);
      const int ch = tid - q + (per == 1 ? 0 : (q >> 1) + (q & 1) * (per / 2));
      const bool direct = a.splits == 1;
#pragma unroll 1
      for (int c0 = 0; c0 < N; c0 += 16) {
        uint32_t o[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) o[r] = 0u;
        if (n > 0) tmem_ld_row<16>(to + c0, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = c0 + i;
          if (sm_t[r] < 0) continue;
          const float lr = sm_w[r] + sm_w[N + r] + sm_w[2 * N + r] + sm_w[3 * N + r];
          const long long row = static_cast<long long>(bh) * n_rows + r0 + r;
          if (!KVQ_IN_BOUNDS(d, kSiteChunkPartial, row, static_cast<long long>(d.B) * d.Hq * a.T)) continue;
          if (direct) {
            a.out[row * kTile + ch] = __float2half_rn(lr > 0.0f ? __uint_as_float(o[i]) / lr : 0.0f);   // sees nothing: 0
          } else {
            const long long part = row * a.splits + split;
            a.o[part * kTile + ch] = __uint_as_float(o[i]);
            if (tid == 0) a.ml[part] = make_float2(lr > 0.0f ? sm_m[r] : -INFINITY, lr);
          }
        }
      }
    }
    fence_before();
  }
  __syncthreads();
  if (warp == 0) {
    fence_after();
    tmem_free(tmem, Lay::kTmem);
  }
}

template <int DK, int N>
cudaError_t launch(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  using Lay = Layout<DK, N>;
  const int stages = ring_stages(d, Lay::kFixed);
  const int smem = Lay::kFixed + stages * ring_stage_bytes(d.kb, d.vb, d.dk);
  static SmemLimit limit;
  const cudaError_t e = limit.raise(chunk_narrow_kernel<DK, N>, smem);
  if (e != cudaSuccess) return e;
  const int row_blocks = (d.n_rep * a.T + N - 1) / N;
  chunk_narrow_kernel<DK, N><<<dim3(a.splits * row_blocks, d.Hkv, d.B), Lay::kThreads, smem, s>>>(d, c, a, stages);
  return cudaGetLastError();
}

template <int DK>
cudaError_t launch_dk(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  return d.n_rep * a.T <= 16 ? launch<DK, 16>(d, c, a, s) : launch<DK, 32>(d, c, a, s);
}

}  // namespace

cudaError_t launch_chunk_narrow(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  return d.dk == 32 ? launch_dk<32>(d, c, a, s) : d.dk == 64 ? launch_dk<64>(d, c, a, s) : launch_dk<128>(d, c, a, s);
}

}  // namespace kvq
