// Chunk attention on the tensor cores (tcgen05, sm_100a), many query rows: flash attention of up
// to 256 rows of a kv head over a packed cache and the new tokens.
//
// A CTA takes one split of the tokens of one (b, kv head, row block), in tiles of 128 tokens (see
// chunk_tile.cuh).  The kv head's n_rep * T query rows are contiguous, so GQA heads and tokens
// fill the 128 MMA rows together and share every decoded key and value.  Roles:
//
//   producers (8 warps)   decode token tiles to fp16 in shared memory;
//   streams (2 x 4 warps) each owns a TMEM tile S/P and an accumulator O.  One of its threads
//                         issues S = Q K^T (operands in shared memory) and O += P V (P in TMEM);
//                         all of them do the softmax, a row per thread, so maxima and sums need
//                         no shuffles.  While one stream's threads work on its tile the tensor
//                         core works for the other.  With up to 128 rows the streams take
//                         alternate token tiles (merged at the end); with more, one row tile each.
//
// Roundings to fp16, each once: decoded keys and values (the MMA's operand type) and the softmax
// weights.  Weights are 2^(s - m + 7) with m a running reference that moves only when a score
// passes it by more than 8, so they stay below 2^15 and are normal numbers down to 2^-21 of the
// largest.  Sums, maxima and O are fp32.
//
// Bound: a tile and row tile cost 2 x 128^3 MMA work, 128^2 exponentials and the decoding of
// 2 x 128 x 128 codes, all three within a factor of two of each other.
#include <algorithm>

#include "chunk_tile.cuh"

namespace kvq {
namespace {

using namespace chunk;

constexpr int kSoftmaxThreads = 256;          // two streams of four warps
constexpr int kThreads = kSoftmaxThreads + kProducers;    // 16 warps: 128 registers a thread

template <int DK, int MT>
struct Layout {
  static constexpr int KH = DK > 64 ? DK / 64 : 1;       // 64-channel halves of a key row
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + MT * KH * kHalf;
  static constexpr int kV = kK + 2 * KH * kHalf;
  static constexpr int kBars = kV + 2 * 2 * kHalf;
  static constexpr int kPages = kBars + 192;
  static constexpr int kMl = kPages + 64;                 // (m, l) of stream 1, for the merge
  static constexpr int kRing = kMl + (MT == 1 ? kTile * 8 : 0);
  static constexpr int kFixed = kRing + 1024;             // the base is aligned to 1024 by hand
  // the merge's copy of stream 1's accumulator (rows of 528 bytes) lies over the K and V stages
  static_assert(MT == 2 || kBars - kK >= kTile * 528, "merge area");
};

enum Bars { kSFull = kTokenBars, kODone = kSFull + 2 };

// One thread: S = Q K^T of a (stream, tile), and O (+)= P V.
template <int DK, int MT>
__device__ __forceinline__ void issue_s(uint32_t base, uint32_t tmem, int stream, int st) {
  using Lay = Layout<DK, MT>;
  const uint32_t q = base + Lay::kQ + (MT == 2 ? stream : 0) * Lay::KH * kHalf;
  const uint32_t k = base + Lay::kK + st * Lay::KH * kHalf;
#pragma unroll
  for (int s = 0; s < DK / 16; ++s) {
    const uint32_t off = (s >> 2) * kHalf + (s & 3) * 32;
    mma_ss(tmem + stream * kTile, desc_sw128(q + off, 16), desc_sw128(k + off, 16), instr_desc(kTile, false, false), s > 0);
  }
}
template <int DK, int MT>
__device__ __forceinline__ void issue_pv(uint32_t base, uint32_t tmem, int stream, int st, bool acc) {
  const uint32_t v = base + Layout<DK, MT>::kV + st * 2 * kHalf;
#pragma unroll
  for (int s = 0; s < kTile / 16; ++s)
    mma_ts(tmem + 2 * kTile + stream * kTile, tmem + stream * kTile + 8 * s, desc_sw128(v + s * 2048, kHalf), instr_desc(kTile, false, true),
           acc || s > 0);
}

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) { return static_cast<uint64_t>(hi) << 32 | lo; }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The streams take turns at the exponentials (every tile: 128 of a row, a thread's longest stretch and
// the special-function unit's).  Side by side they would both crawl through them and then both wait
// for the tensor core; in turn one computes weights while the other's products run.
__device__ __forceinline__ void turn_take(int stream) {
  if (stream == 0)
    asm volatile("bar.sync 5, 256;" ::: "memory");
  else
    asm volatile("bar.sync 6, 256;" ::: "memory");
}
__device__ __forceinline__ void turn_pass(int stream) {
  if (stream == 0)
    asm volatile("bar.arrive 6, 256;" ::: "memory");
  else
    asm volatile("bar.arrive 5, 256;" ::: "memory");
}

// The scores of 64 columns that a row does not see become -inf.
__device__ __forceinline__ void mask64(uint32_t (&x)[64], uint32_t see0, uint32_t see1) {
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (!((i < 32 ? see0 : see1) >> (i & 31) & 1u)) x[i] = 0xff800000u;
}
__device__ __forceinline__ float max64(const uint32_t (&x)[64], float m) {
  float m4[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 64; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(x[i]));
  return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
}
// p = 2^(x alpha + off) of 64 columns to 32 TMEM columns of fp16 pairs; returns their sum.
__device__ __forceinline__ float weights64(const uint32_t (&x)[64], float alpha, float off, uint32_t dst) {
  const uint64_t a2 = pack2(__float_as_uint(alpha), __float_as_uint(alpha));
  const uint64_t o2 = pack2(__float_as_uint(off), __float_as_uint(off));
  uint64_t l2[2] = {0ull, 0ull};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint64_t e = fma2(pack2(x[32 * h + 2 * i], x[32 * h + 2 * i + 1]), a2, o2);
      const float p0 = ptx::ex2(__uint_as_float(static_cast<uint32_t>(e)));
      const float p1 = ptx::ex2(__uint_as_float(static_cast<uint32_t>(e >> 32)));
      l2[i & 1] = add2(l2[i & 1], pack2(__float_as_uint(p0), __float_as_uint(p1)));
      p[i] = ptx::h2_as_u32(__floats2half2_rn(p0, p1));
    }
    tmem_st16(dst + 16 * h, p);
  }
  const uint64_t l = add2(l2[0], l2[1]);
  return __uint_as_float(static_cast<uint32_t>(l)) + __uint_as_float(static_cast<uint32_t>(l >> 32));
}

template <int VB>
__device__ __forceinline__ void store_row(const uint32_t (&x)[32], float f, __half* out, float* part) {
  if (out) {
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = ptx::h2_as_u32(__floats2half2_rn(__uint_as_float(x[column_of<VB>(i + 2 * e)]) * f,
                                                __uint_as_float(x[column_of<VB>(i + 2 * e + 1)]) * f));
      *reinterpret_cast<uint4*>(out + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      *reinterpret_cast<float4*>(part + i) =
          make_float4(__uint_as_float(x[column_of<VB>(i)]) * f, __uint_as_float(x[column_of<VB>(i + 1)]) * f,
                      __uint_as_float(x[column_of<VB>(i + 2)]) * f, __uint_as_float(x[column_of<VB>(i + 3)]) * f);
  }
}

template <int DK, int MT>
__global__ void __launch_bounds__(kThreads, 1)
chunk_wide_kernel(const __grid_constant__ Dims d, const __grid_constant__ CacheBufs cb,
                 const __grid_constant__ ChunkArgs a, int stages) {
  using Lay = Layout<DK, MT>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  __shared__ uint32_t sm_tmem;
  __shared__ int sm_fail;

  const int split = blockIdx.x % a.splits, rb = blockIdx.x / a.splits, h = blockIdx.y, b = blockIdx.z;
  const int bh = b * d.Hkv + h;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const SeqNew s = seq_new(a.seq, b, d.log_retain);
  const int n_rows = d.n_rep * a.T, r0 = rb * MT * kTile;

  Tiles t;
  if (!block_tiles(a, s, r0, min(r0 + MT * kTile, n_rows) - 1, split, t)) return;
  const int n = t.end - t.begin;

  const uint32_t bars = base + Lay::kBars;
  if (tid == 0) {
    init_token_bars(bars, kProducers / 32, kProducers / 32, MT);   // with two row tiles both streams use a tile
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars + 8 * (kSFull + i), 1);
      ptx::mbar_init(bars + 8 * (kODone + i), 1);
    }
    ptx::fence_barrier_init();
    sm_fail = 0;
  }
  clear_ring(d, base + Lay::kRing, stages, tid, kThreads);
  if (warp == 0) tmem_alloc(ptx::smem_addr(&sm_tmem), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm_tmem;
  const Waiter wait{&sm_fail};

  float m_ref = -INFINITY, l = 0.0f;
  const int stream = (warp >> 2) & 1;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const int row = r0 + (MT == 2 ? stream * kTile : 0) + (tid & 127);       // this softmax thread's row of the block
  const int tr = row % a.T;
  const bool row_ok = row < n_rows && tr < s.n;
  int mine = 0;                                                            // tiles this stream took

  if (warp >= kSoftmaxThreads / 32) {
    const int pt = tid - kSoftmaxThreads;
    const Ctx c{d, cb, a, s, b, h, bh, __ffs(d.gk) - 1, __ffs(d.gv) - 1, __ffs(d.nvg) - 1,
                base + Lay::kRing, base + Lay::kPages, stages};
    with_bits(d, [&](auto kb, auto vb) {
      for (int i = 0; i < MT; ++i)
        copy_queries<kb.value, DK, kTile>(c, r0 + i * kTile, n_rows, pt, base + Lay::kQ + i * Lay::KH * kHalf);
      produce<kb.value, vb.value, DK, true>(c, t, pt, base + Lay::kK, base + Lay::kV, bars, wait);
    });
  } else {
    const uint32_t ts = tmem + stream * kTile + lanes, to = tmem + 2 * kTile + stream * kTile + lanes;
    const int ret_pos = lane < s.n_ret ? retained_position(s.Q, lane) : -1;
    const int mask_words = (a.T + 31) / 32;
    const float alpha = a.score_scale;
    constexpr int kStride = MT == 2 ? 1 : 2;
    const int first = MT == 2 ? 0 : stream;
    const bool issuer = (warp & 3) == 0;       // the stream's first warp
    const bool idle = !__any_sync(0xffffffffu, row_ok);       // no row of the warp counts: P may be anything
    if (stream == 1) turn_pass(1);          // stream 0 begins
    bool live = true;
    // S of the stream's tile `it`, once its keys are there
    auto score = [&](int it) {
      const int st = it & 1;
      if (!__all_sync(0xffffffffu, wait(bars + 8 * (kKFull + st), (it >> 1) & 1))) return;
      fence_after();
      __syncwarp();
      if (elect_one()) {
        issue_s<DK, MT>(base, tmem, stream, st);
        commit(bars + 8 * (kSFull + stream));
        commit(bars + 8 * (kKEmpty + st));
      }
      __syncwarp();
    };
    if (issuer && first < n) score(first);
    for (int it = first; it < n; it += kStride, ++mine) {
      // a wait that runs out ends the work, not the loop: the stream's barrier counts every warp
      live = live && __all_sync(0xffffffffu, wait(bars + 8 * (kSFull + stream), mine & 1));
      fence_after();
      bool full = true;
      uint32_t see[4];                       // columns of the tile the row sees, 32 a word (unless `full`)
      if (live && !idle) {
        const int tile = t.begin + it;
        const int kind = tile < t.nq ? 0 : tile < t.nq + t.nf ? 1 : 2;
        const int e0 = (tile - (kind > 0 ? t.nq : 0) - (kind > 1 ? t.nf : 0)) * kTile;
        const int nv = (kind == 0 ? s.Q : kind == 1 ? t.n_fp16 : t.n_vis) - e0;
        // retained tokens of a quantized tile are read from the fp16 list
        unsigned hits = 0u;
        if (kind == 0 && s.n_ret) hits = __ballot_sync(0xffffffffu, ret_pos >= e0 && ret_pos < e0 + kTile);
        full = nv >= kTile && hits == 0 && kind != 2;
        if (!full) {
#pragma unroll
          for (int c = 0; c < 4; ++c) see[c] = below(nv - 32 * c);
          while (hits) {
            const int off = __shfl_sync(0xffffffffu, ret_pos, __ffs(hits) - 1) - e0;
            hits &= hits - 1;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (off >> 5 == c) see[c] &= ~(1u << (off & 31));
          }
          if (kind == 2) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int j0 = e0 + 32 * c;
              if (!a.mask)
                see[c] &= below(tr + 1 - j0);
              else
                see[c] &= row_ok && j0 < a.T ? a.mask[(static_cast<long long>(b) * a.T + tr) * mask_words + j0 / 32] : 0u;
            }
            full = __all_sync(0xffffffffu, (see[0] & see[1] & see[2] & see[3]) == 0xffffffffu);
          }
        }
      }
      if (live && !idle) {
        float mx = -INFINITY;
#pragma unroll 1
        for (int h2 = 0; h2 < 2; ++h2) {      // loops, not copies: the roles' code shares an instruction cache
          uint32_t x[64];
          tmem_ld64(ts + 64 * h2, x);
          tmem_wait_ld();
          if (!full) mask64(x, h2 ? see[2] : see[0], h2 ? see[3] : see[1]);
          mx = max64(x, mx);
        }
        const float m_new = mx * alpha;
        const bool mv = m_new > m_ref + kLazy;
        if (__any_sync(0xffffffffu, mv)) {
          const float f = mv ? ptx::ex2(m_ref - m_new) : 1.0f;
          if (mv) m_ref = m_new;
          l *= f;
          // S of this tile is committed behind the stream's last P V, so O is complete
          if (mine > 0) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(to + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st32(to + 32 * c, o);
            }
          }
        }
      }
      turn_take(stream);
      if (live && !idle) {
        const float off = kBias - (m_ref == -INFINITY ? 0.0f : m_ref);
        // the weights of a half's columns go to 32 columns whose scores have been read
#pragma unroll 1
        for (int h2 = 0; h2 < 2; ++h2) {
          uint32_t x[64];
          tmem_ld64(ts + 64 * h2, x);
          tmem_wait_ld();
          if (!full) mask64(x, h2 ? see[2] : see[0], h2 ? see[3] : see[1]);
          l += weights64(x, alpha, off, ts + 32 * h2);
        }
        tmem_wait_st();
      }
      turn_pass(stream);
      fence_before();
      if (stream == 0)
        asm volatile("bar.sync 2, 128;" ::: "memory");
      else
        asm volatile("bar.sync 3, 128;" ::: "memory");
      if (issuer && live) {
        const int st = it & 1;
        if (__all_sync(0xffffffffu, wait(bars + 8 * (kVFull + st), (it >> 1) & 1))) {
          fence_after();
          if (elect_one()) {
            issue_pv<DK, MT>(base, tmem, stream, st, mine > 0);
            commit(bars + 8 * (kVEmpty + st));
          }
          __syncwarp();
          if (it + kStride < n) score(it + kStride);
        }
      }
      __syncwarp();
    }
    if (mine > 0) {
      // everything issued has to end before the CTA reuses its memory or frees its TMEM, also
      // after a wait that ran out
      if (issuer && elect_one()) commit(bars + 8 * (kODone + stream));
      __syncwarp();
      if (!ptx::mbar_wait_bounded(bars + 8 * (kODone + stream), 0, kWaitNs)) *wait.fail = 1;
      fence_after();
    }
  }
  __syncthreads();
  const bool failed = sm_fail != 0;
  if (failed && tid == 0) atomicOr(a.status, KVQ_STATUS_TIMEOUT);

  // ---------------- outputs ----------------
  if (warp < 8 && !failed) {
    const uint32_t to = tmem + 2 * kTile + stream * kTile + lanes;
    float2* sm_ml = reinterpret_cast<float2*>(smem + Lay::kMl);
    unsigned char* merge = smem + Lay::kK;
    float w0 = 1.0f, w1 = 0.0f;
    if constexpr (MT == 1) {
      // stream 1 hands its accumulator to stream 0
      if (stream == 1) {
        sm_ml[tid & 127] = make_float2(m_ref, l);
        if (mine > 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32(to + 32 * c, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(merge + (tid & 127) * 528 + (32 * c + i) * 4) =
                  make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          }
        }
      }
      asm volatile("bar.sync 4, %0;" ::"n"(kSoftmaxThreads) : "memory");
      if (stream == 0) {
        const float2 o = sm_ml[tid & 127];
        const float M = fmaxf(m_ref, o.x);
        w0 = m_ref == -INFINITY ? 0.0f : ptx::ex2(m_ref - M);
        w1 = o.x == -INFINITY ? 0.0f : ptx::ex2(o.x - M);
        l = l * w0 + o.y * w1;
        m_ref = M;
      }
    }
    if (MT == 2 || stream == 0) {
      const long long orow = static_cast<long long>(bh) * n_rows + row, part = orow * a.splits + split;
      const bool direct = a.splits == 1;
      const float f = direct ? (l > 0.0f ? 1.0f / l : 0.0f) : 1.0f;      // a row that sees nothing: 0
      const bool pok = KVQ_IN_BOUNDS(d, kSiteChunkPartial, row_ok ? orow : 0, static_cast<long long>(d.B) * d.Hq * a.T);
      if (!direct && row_ok && pok) a.ml[part] = make_float2(m_ref, l);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        if (n > 0) {
          tmem_ld32(to + 32 * c, x);
          tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float v = n > 0 && l > 0.0f ? __uint_as_float(x[i]) * w0 : 0.0f;
          if (MT == 1 && n > 1 && w1 != 0.0f)
            v = fmaf(*reinterpret_cast<const float*>(merge + (tid & 127) * 528 + (32 * c + i) * 4), w1, v);
          x[i] = __float_as_uint(v);
        }
        if (row_ok && pok) {
          __half* out = direct ? a.out + orow * kTile + 32 * c : nullptr;
          float* po = direct ? nullptr : a.o + part * kTile + 32 * c;
          switch (d.vb) {
            case 2: store_row<2>(x, f, out, po); break;
            case 4: store_row<4>(x, f, out, po); break;
            case 8: store_row<8>(x, f, out, po); break;
            default: store_row<16>(x, f, out, po); break;
          }
        }
      }
    }
    fence_before();
  }
  __syncthreads();
  if (warp == 0) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

template <int DK, int MT>
cudaError_t launch(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  const int stages = ring_stages(d, Layout<DK, MT>::kFixed);
  const int smem = Layout<DK, MT>::kFixed + stages * ring_stage_bytes(d.kb, d.vb, d.dk);
  static SmemLimit limit;
  const cudaError_t e = limit.raise(chunk_wide_kernel<DK, MT>, smem);
  if (e != cudaSuccess) return e;
  const int row_blocks = (d.n_rep * a.T + MT * kTile - 1) / (MT * kTile);
  chunk_wide_kernel<DK, MT><<<dim3(a.splits * row_blocks, d.Hkv, d.B), kThreads, smem, s>>>(d, c, a, stages);
  return cudaGetLastError();
}

// Row tiles of a CTA: two where there are rows for them and the second one's queries leave room for
// a stage of the packed ring (at d_k 128 all but 8-bit keys with 8-bit values).
int row_tiles(const Dims& d, int T) {
  if (d.n_rep * T <= kTile) return 1;
  const int used = d.dk == 32 ? Layout<32, 2>::kFixed : d.dk == 64 ? Layout<64, 2>::kFixed : Layout<128, 2>::kFixed;
  return !d.quantized() || ring_stages(d, used) > 0 ? 2 : 1;
}

}  // namespace

bool chunk_mma_supported(const Dims& d) {
  if (d.var || d.sr || d.dv != kTile || d.dk > 128) return false;
  if (!d.quantized()) return true;
  return d.gk >= 32 && d.gv >= 32;
}

int chunk_mma_splits(const Dims& d, int L, int T, int num_splits) {
  const int tiles = (L + T + kTile - 1) / kTile + 1;
  if (num_splits > 0) return std::min({num_splits, tiles, 64});
  // waves of one CTA per SM: a CTA costs its tiles and about three more (launch, first tile, epilogue)
  const int rows = d.n_rep * T, block = rows > kNarrowRows ? row_tiles(d, T) * kTile : rows;
  const long long units = static_cast<long long>(d.B) * d.Hkv * ((rows + block - 1) / block);
  int best = 1;
  double best_t = 1e300;
  for (int s = 1; s <= std::min(tiles, 64); ++s) {
    const double t = static_cast<double>((units * s + d.sm_count - 1) / d.sm_count) * ((tiles + s - 1) / s + 3.0);
    if (t < best_t * 0.98) {
      best_t = t;
      best = s;
    }
  }
  return best;
}

cudaError_t launch_chunk_mma(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  if (d.n_rep * a.T <= kNarrowRows) return launch_chunk_narrow(d, c, a, s);
  const bool wide = row_tiles(d, a.T) == 2;
  switch (d.dk) {
    case 32: return wide ? launch<32, 2>(d, c, a, s) : launch<32, 1>(d, c, a, s);
    case 64: return wide ? launch<64, 2>(d, c, a, s) : launch<64, 1>(d, c, a, s);
    default: return wide ? launch<128, 2>(d, c, a, s) : launch<128, 1>(d, c, a, s);
  }
}

}  // namespace kvq
