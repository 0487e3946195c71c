// Chunk attention on the tensor cores (tcgen05, sm_100a): flash attention of up to 256 query
// rows of a kv head over a packed cache and the new tokens.
//
// A CTA takes one split of the tokens of one (b, kv head, row block), in tiles of 128 tokens:
// the quantized prefix, the fp16 list (retained tokens, window), the new tokens.  The kv head's
// n_rep * T query rows are contiguous, so GQA heads and tokens fill the 128 MMA rows together
// and share every decoded key and value.  Roles, all in flight at once:
//
//   producers (8 warps)  read packed codes (registers, one tile ahead) and their (scale, zero)
//                        (cp.async, one tile ahead), decode to fp16 and write the tile to shared
//                        memory in the 128-byte swizzle the MMA reads: keys K-major, values
//                        MN-major, a token per 128-byte row in both.
//   MMA (1 thread)       S = Q K^T (both operands in shared memory), then O += P V (P in TMEM).
//   softmax (2 x 4 warps) two independent streams, each a TMEM tile S/P and an accumulator O:
//                        a thread owns a row, so maxima and sums need no shuffles.  With up to
//                        128 rows the streams take alternate token tiles (merged at the end);
//                        with more, one row tile each.
//
// A key code pair masked out of a packed word sits in the two halves of a register, so decoding
// yields channels (i, i + 16/bits) next to each other; the channel order of a dot product is
// free, so Q is laid out in that order, and the outputs' order is undone in the epilogue.  Per
// pair: one LOP3 (1024 + code), one exact subtraction, one fused multiply-add that rounds
// code * s + z to fp16 once.
//
// Roundings to fp16, each once: decoded keys and values (the MMA's operand type; the codes
// themselves carry at most 8 bits) and the softmax weights.  Weights are 2^(s - m + 7) with m a
// running reference that moves only when a score passes it by more than 8, so they stay below
// 2^15 and are normal numbers down to 2^-21 of the largest.  Sums, maxima and O are fp32.
//
// Bound: at 128 rows the tile costs 2 x 128^3 MMA work, 128^2 exponentials and the decoding of
// 2 x 128 x 128 codes, all three within a factor of two of each other; with few rows it is the
// same work on padded rows.
#include <algorithm>

#include "../../include/kvq.h"
#include "ptx.cuh"
#include "seq_ops.cuh"

namespace kvq {
namespace {

constexpr int kSoftmaxThreads = 256;          // two streams of four warps
constexpr int kProducerThreads = 256;
constexpr int kProducerWarps = kProducerThreads / 32;
constexpr int kThreads = kSoftmaxThreads + kProducerThreads + 32;
constexpr int kTile = 128;                    // tokens per tile, rows per row tile, value channels
constexpr int kHalf = kTile * 128;            // bytes of 128 rows of 64 fp16 channels
constexpr int kMetaStage = 4096;              // (scale, zero) of a tile: keys 2 KB, values 2 KB
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kLazy = 8.0f;                 // log2 units the reference maximum may lag
constexpr float kBias = 7.0f;                 // weights are 2^(s - m + kBias) < 2^15

// ---- tcgen05 ----
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"(static_cast<uint32_t>(acc))
      : "memory");
}
#define KVQ_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define KVQ_W4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KVQ_R4(r, 0), KVQ_R4(r, 4), KVQ_R4(r, 8), KVQ_R4(r, 12), KVQ_R4(r, 16), KVQ_R4(r, 20), KVQ_R4(r, 24), KVQ_R4(r, 28)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::KVQ_W4(r, 0), KVQ_W4(r, 4), KVQ_W4(r, 8),
      KVQ_W4(r, 12), KVQ_W4(r, 16), KVQ_W4(r, 20), KVQ_W4(r, 24), KVQ_W4(r, 28), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::KVQ_W4(
          r, 0), KVQ_W4(r, 4), KVQ_W4(r, 8), KVQ_W4(r, 12), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major (Q, K): 8-row groups 1024 bytes
// apart.  MN-major (V): 8-token groups 1024 bytes apart, 64-channel halves kHalf apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | static_cast<uint64_t>(lbo >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
constexpr uint32_t kIdesc = 1u << 4 | (kTile / 8) << 17 | (kTile / 16) << 24;   // f16 x f16 -> f32, 128 x 128
constexpr uint32_t kIdescPV = kIdesc | 1u << 16;                                // B (values) MN-major

template <int DK, int MT>
struct Layout {
  static constexpr int KH = DK > 64 ? DK / 64 : 1;       // 64-channel halves of a key row
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + MT * KH * kHalf;
  static constexpr int kV = kK + 2 * KH * kHalf;
  static constexpr int kMeta = kV + 2 * 2 * kHalf;
  static constexpr int kBars = kMeta + 2 * kMetaStage;
  static constexpr int kMl = kBars + 256;                 // (m, l) of stream 1, for the merge
  static constexpr int kBytes = kMl + kTile * 8 + 1024;   // the base is aligned to 1024 by hand
  // the merge's copy of stream 1's accumulator (rows of 528 bytes) lies over the K and V stages
  static_assert(MT == 2 || kMeta - kK >= kTile * 528, "merge area");
};

enum Bars { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPFull = 10, kODone = 12, kNumBars = 13 };

// ---- the token tiles of a CTA ----
struct Tiles {
  int nq, nf, begin, end;     // quantized tiles, fp16-list tiles; this CTA's range of all tiles
  int n_fp16, n_vis;          // entries of the fp16 list; new tokens that some row of the block may see
};

// Channel pair order: position 2i, 2i + 1 of a block of 32 / bits channels is channel i, i + 16 / bits.
template <int BITS>
__device__ __forceinline__ void permute32(uint4& x, uint4& y) {
  if constexpr (BITS == 8) {
    const uint4 a = x, b = y;
    x = make_uint4(ptx::prmt(a.x, a.y, 0x5410), ptx::prmt(a.x, a.y, 0x7632), ptx::prmt(a.z, a.w, 0x5410),
                   ptx::prmt(a.z, a.w, 0x7632));
    y = make_uint4(ptx::prmt(b.x, b.y, 0x5410), ptx::prmt(b.x, b.y, 0x7632), ptx::prmt(b.z, b.w, 0x5410),
                   ptx::prmt(b.z, b.w, 0x7632));
  } else if constexpr (BITS == 4) {
    const uint4 a = x, b = y;
    x = make_uint4(ptx::prmt(a.x, a.z, 0x5410), ptx::prmt(a.x, a.z, 0x7632), ptx::prmt(a.y, a.w, 0x5410),
                   ptx::prmt(a.y, a.w, 0x7632));
    y = make_uint4(ptx::prmt(b.x, b.z, 0x5410), ptx::prmt(b.x, b.z, 0x7632), ptx::prmt(b.y, b.w, 0x5410),
                   ptx::prmt(b.y, b.w, 0x7632));
  } else if constexpr (BITS == 2) {
    const uint4 a = x, b = y;
    x = make_uint4(ptx::prmt(a.x, b.x, 0x5410), ptx::prmt(a.x, b.x, 0x7632), ptx::prmt(a.y, b.y, 0x5410),
                   ptx::prmt(a.y, b.y, 0x7632));
    y = make_uint4(ptx::prmt(a.z, b.z, 0x5410), ptx::prmt(a.z, b.z, 0x7632), ptx::prmt(a.w, b.w, 0x5410),
                   ptx::prmt(a.w, b.w, 0x7632));
  }
}

// 16-byte chunk j (8 channels) of row t of a tile of 128-byte rows in the 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_at(int t, int j) {
  return (j >> 3) * kHalf + t * 128 + (((j & 7) ^ (t & 7)) << 4);
}
__device__ __forceinline__ void st_shared(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// The code pair in field I (bits I * BITS of both halves of w), as exact fp16 values.
template <int BITS, int I>
__device__ __forceinline__ __half2 code_pair(uint32_t w) {
  constexpr int shift = (BITS * I) / 8 * 8, low = BITS * I - shift;     // byte shift, then bit offset below 8
  constexpr uint32_t mask = ((1u << BITS) - 1u) * 0x00010001u << low;
  const uint32_t x = ((w >> shift) & mask) | 0x64006400u;               // 1024 + code * 2^low
  if constexpr (low == 0) return __hsub2(ptx::u32_as_h2(x), __float2half2_rn(1024.0f));
  constexpr float inv = 1.0f / (1 << low);
  return __hfma2(ptx::u32_as_h2(x), __float2half2_rn(inv), __float2half2_rn(-1024.0f * inv));
}
template <int BITS, int I>
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, uint32_t s, uint32_t z) {
  return ptx::h2_as_u32(__hfma2(code_pair<BITS, I>(w), ptx::u32_as_h2(s), ptx::u32_as_h2(z)));
}

// A thread's share of a tile's packed keys: unit u of the row (a chunk of 8 channels, or 16 at 2
// bits), tokens sub, sub + kStep, ...
template <int KB, int DK>
struct KeyUnits {
  static constexpr int kPerRow = KB == 2 ? DK / 16 : DK / 8;
  static constexpr int kWords = KB == 8 ? 2 : 1;
  static constexpr int kStep = kProducerThreads / kPerRow;
  static constexpr int kTokens = kTile / kStep;
};

// Everything the producers share.
struct Ctx {
  const Dims& d;
  const CacheBufs& cb;
  const ChunkArgs& a;
  const SeqNew& s;
  int b, h, bh;
};

__device__ __forceinline__ long long token_row(const Ctx& c, int p) {
  const int g = p / c.d.gk;
  if (!KVQ_IN_BOUNDS(c.d, kSiteChunkTable, g, c.d.max_groups)) return 0;
  long long row = static_cast<long long>(group_row(c.d, c.cb.table, c.b, c.h, g)) + (p & (c.d.gk - 1));
  if (!KVQ_IN_BOUNDS(c.d, kSiteChunkRow, row, quant_rows(c.d))) row = 0;
  return row;
}

template <int KB, int DK>
__device__ __forceinline__ void load_key_codes(const Ctx& c, int p0, int tid, uint32_t* w) {
  using U = KeyUnits<KB, DK>;
  const int u = tid % U::kPerRow, sub = tid / U::kPerRow;
#pragma unroll
  for (int i = 0; i < U::kTokens; ++i) {
    const int p = p0 + sub + i * U::kStep;
#pragma unroll
    for (int k = 0; k < U::kWords; ++k) w[i * U::kWords + k] = 0u;
    if (p < c.s.Q) {
      const uint32_t* src = c.cb.kcode + token_row(c, p) * (DK * KB / 32) + u * U::kWords;
      if constexpr (U::kWords == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
        w[2 * i] = x.x;
        w[2 * i + 1] = x.y;
      } else {
        w[i] = __ldg(src);
      }
    }
  }
}

// The thread's codes to fp16 rows of the key tile at `dst`; meta: the groups' (scale, zero) blocks.
template <int KB, int DK>
__device__ __forceinline__ void decode_keys(const Ctx& c, int p0, int tid, const uint32_t* w, uint32_t meta,
                                            uint32_t dst) {
  using U = KeyUnits<KB, DK>;
  constexpr int P = 32 / KB, W = DK / P;
  const int u = tid % U::kPerRow, sub = tid / U::kPerRow;
  const int lgk = __ffs(c.d.gk) - 1;
  auto pos = [](int wd) { return W % 4 == 0 ? (wd % (W / 4)) * 4 + wd / (W / 4) : wd; };
  // (scale, zero) pairs of the unit, reloaded when the group changes: s[i], z[i] of register i
  constexpr int R = U::kWords * P / 2;
  uint32_t sc[R], zr[R];
  int cur = -1;
#pragma unroll
  for (int i = 0; i < U::kTokens; ++i) {
    const int t = sub + i * U::kStep, g = t >> lgk;
    const bool valid = p0 + t < c.s.Q;
    if (g != cur) {
      cur = g;
#pragma unroll
      for (int k = 0; k < U::kWords; ++k) {
        const uint32_t at = meta + g * (DK * 4) + pos(u * U::kWords + k) * (4 * P);
#pragma unroll
        for (int e = 0; e < P; e += 4) {       // P registers: P / 2 scale pairs, then P / 2 zero pairs
          const uint4 m = ld_shared(at + 4 * e);
          const uint32_t mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            if (e + f < P / 2)
              sc[k * (P / 2) + e + f] = mm[f];
            else
              zr[k * (P / 2) + e + f - P / 2] = mm[f];
          }
        }
      }
    }
    uint32_t o[R];
    if constexpr (KB == 8) {
      o[0] = decode_pair<8, 0>(w[2 * i], sc[0], zr[0]);
      o[1] = decode_pair<8, 1>(w[2 * i], sc[1], zr[1]);
      o[2] = decode_pair<8, 0>(w[2 * i + 1], sc[2], zr[2]);
      o[3] = decode_pair<8, 1>(w[2 * i + 1], sc[3], zr[3]);
    } else if constexpr (KB == 4) {
      o[0] = decode_pair<4, 0>(w[i], sc[0], zr[0]);
      o[1] = decode_pair<4, 1>(w[i], sc[1], zr[1]);
      o[2] = decode_pair<4, 2>(w[i], sc[2], zr[2]);
      o[3] = decode_pair<4, 3>(w[i], sc[3], zr[3]);
    } else {
      o[0] = decode_pair<2, 0>(w[i], sc[0], zr[0]);
      o[1] = decode_pair<2, 1>(w[i], sc[1], zr[1]);
      o[2] = decode_pair<2, 2>(w[i], sc[2], zr[2]);
      o[3] = decode_pair<2, 3>(w[i], sc[3], zr[3]);
      o[4] = decode_pair<2, 4>(w[i], sc[4], zr[4]);
      o[5] = decode_pair<2, 5>(w[i], sc[5], zr[5]);
      o[6] = decode_pair<2, 6>(w[i], sc[6], zr[6]);
      o[7] = decode_pair<2, 7>(w[i], sc[7], zr[7]);
    }
#pragma unroll
    for (int e = 0; e < R; e += 4) {
      const uint4 v = valid ? make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_uint4(0, 0, 0, 0);
      st_shared(dst + chunk_at(t, u * (R / 4) + e / 4), v);
    }
  }
}

// Values: thread (token tid / 2, channel half tid % 2) decodes 64 channels.  The halves take
// their eight chunks in opposite order, so that the eight threads of a store phase (four tokens,
// both halves) write eight different bank groups.
template <int VB>
__device__ __forceinline__ void load_value_codes(const Ctx& c, int p0, int tid, uint32_t* w) {
  constexpr int N = 2 * VB;      // words of 64 channels
  const int p = p0 + (tid >> 1), half = tid & 1;
#pragma unroll
  for (int k = 0; k < N; ++k) w[k] = 0u;
  if (p < c.s.Q) {
    const uint4* src = reinterpret_cast<const uint4*>(c.cb.vcode + token_row(c, p) * (4 * VB) + half * N);
    const int flip = half ? N / 8 : 0;          // chunk order 4..7, 0..3 for the second half
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      if constexpr (VB == 2) {
        const uint4 x = __ldg(src);
        w[0] = half ? x.z : x.x;
        w[1] = half ? x.w : x.y;
        w[2] = half ? x.x : x.z;
        w[3] = half ? x.y : x.w;
      } else {
        const uint4 x = __ldg(src + (k ^ flip));
        w[4 * k] = x.x;
        w[4 * k + 1] = x.y;
        w[4 * k + 2] = x.z;
        w[4 * k + 3] = x.w;
      }
    }
  }
}

template <int VB>
__device__ __forceinline__ void decode_values(const Ctx& c, int p0, int tid, const uint32_t* w, uint32_t meta,
                                              uint32_t dst) {
  const int t = tid >> 1, half = tid & 1;
  const bool valid = p0 + t < c.s.Q;
  const int lgv = __ffs(c.d.gv) - 1;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int j = half * 8 + (half ? k ^ 4 : k);                    // chunk of the row: channels 8j .. 8j + 7
    // chunks come in pairs of one (scale, zero): groups hold at least 32 channels
    const uint32_t sz = ld_shared32(meta + (t * c.d.nvg + (8 * j >> lgv)) * 4);
    const uint32_t s = ptx::prmt(sz, sz, 0x1010), z = ptx::prmt(sz, sz, 0x3232);
    uint32_t o[4];
    if constexpr (VB == 8) {
      o[0] = decode_pair<8, 0>(w[2 * k], s, z);
      o[1] = decode_pair<8, 1>(w[2 * k], s, z);
      o[2] = decode_pair<8, 0>(w[2 * k + 1], s, z);
      o[3] = decode_pair<8, 1>(w[2 * k + 1], s, z);
    } else if constexpr (VB == 4) {
      o[0] = decode_pair<4, 0>(w[k], s, z);
      o[1] = decode_pair<4, 1>(w[k], s, z);
      o[2] = decode_pair<4, 2>(w[k], s, z);
      o[3] = decode_pair<4, 3>(w[k], s, z);
    } else if (k % 2 == 0) {
      o[0] = decode_pair<2, 0>(w[k / 2], s, z);
      o[1] = decode_pair<2, 1>(w[k / 2], s, z);
      o[2] = decode_pair<2, 2>(w[k / 2], s, z);
      o[3] = decode_pair<2, 3>(w[k / 2], s, z);
    } else {
      o[0] = decode_pair<2, 4>(w[k / 2], s, z);
      o[1] = decode_pair<2, 5>(w[k / 2], s, z);
      o[2] = decode_pair<2, 6>(w[k / 2], s, z);
      o[3] = decode_pair<2, 7>(w[k / 2], s, z);
    }
    st_shared(dst + chunk_at(t, j), valid ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(0, 0, 0, 0));
  }
}

// The (scale, zero) blocks of a quantized tile, a 16-byte piece per thread: keys by the first
// 128 threads, values by the others.
template <int DK>
__device__ __forceinline__ void fetch_meta(const Ctx& c, int p0, int tid, uint32_t dst) {
  const Dims& d = c.d;
  if (tid < 128) {
    constexpr int pieces = DK / 4;              // per group
    const int gi = tid / pieces, e = tid % pieces, p = p0 + gi * d.gk;
    if (gi * d.gk < kTile && p < c.s.Q) {
      const int g = p / d.gk;
      long long gidx = KVQ_IN_BOUNDS(d, kSiteChunkTable, g, d.max_groups)
                           ? static_cast<long long>(group_index(d, c.cb.table, c.b, c.h, g)) : 0;
      if (!KVQ_IN_BOUNDS(d, kSiteChunkGroup, gidx, quant_groups(d))) gidx = 0;
      cp_async_16(dst + gi * DK * 4 + e * 16, reinterpret_cast<const uint4*>(c.cb.ksz + gidx * DK) + e);
    }
  } else {
    const int e = tid - 128, t = e * 4 / d.nvg;            // four (scale, zero) pairs a piece
    if (t < kTile && p0 + t < c.s.Q)
      cp_async_16(dst + 2048 + e * 16, c.cb.vsz + token_row(c, p0 + t) * d.nvg);
  }
}

// fp16 rows of the list (kind 1) or of the new tokens (kind 2) to a tile; entries from `n` on are zero.
// WIDTH channels a row; the channel order is that of BITS-bit codes.
template <int BITS, int WIDTH>
__device__ __forceinline__ void copy_rows(const Ctx& c, bool keys, int kind, int e0, int n, int tid, uint32_t dst) {
  constexpr int per_row = WIDTH / 16, step = kProducerThreads / per_row, tokens = kTile / step;
  const int u = tid % per_row, sub = tid / per_row;
  const __half* ret = keys ? c.cb.ret_k : c.cb.ret_v;
  const __half* win = keys ? c.cb.win_k : c.cb.win_v;
  const __half* fresh = keys ? c.a.k_new : c.a.v_new;
  uint4 x[tokens], y[tokens];
#pragma unroll
  for (int i = 0; i < tokens; ++i) {
    const int e = e0 + sub + i * step;
    x[i] = y[i] = make_uint4(0, 0, 0, 0);
    if (e < n) {
      const __half* row;
      if (kind == 2) {
        row = fresh + (static_cast<long long>(c.bh) * c.a.T + e) * WIDTH;
      } else if (e < c.s.n_ret) {
        long long r = static_cast<long long>(c.bh) * kMaxRetained + e;
        if (!KVQ_IN_BOUNDS(c.d, kSiteChunkFp16, r, ret_rows(c.d))) r = 0;
        row = ret + r * WIDTH;
      } else {
        long long r = static_cast<long long>(c.bh) * c.d.cap + (c.s.Q + e - c.s.n_ret) % c.d.cap;
        if (!KVQ_IN_BOUNDS(c.d, kSiteChunkFp16, r, win_rows(c.d))) r = 0;
        row = win + r * WIDTH;
      }
      x[i] = __ldg(reinterpret_cast<const uint4*>(row) + 2 * u);
      y[i] = __ldg(reinterpret_cast<const uint4*>(row) + 2 * u + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < tokens; ++i) {
    const int t = sub + i * step;
    permute32<BITS>(x[i], y[i]);
    st_shared(dst + chunk_at(t, 2 * u), x[i]);
    st_shared(dst + chunk_at(t, 2 * u + 1), y[i]);
  }
}

// Query rows r0 .. r0 + 128 of the kv head's block (rows of T tokens per head; those behind the
// sequence's new tokens are zero), in the keys' channel order.
template <int KB, int DK>
__device__ __forceinline__ void copy_queries(const Ctx& c, int r0, int n_rows, int tid, uint32_t dst) {
  constexpr int per_row = DK / 16, step = kProducerThreads / per_row;
  const int u = tid % per_row, sub = tid / per_row;
  const __half* q = c.a.q + static_cast<long long>(c.bh) * n_rows * DK;
  for (int t = sub; t < kTile; t += step) {
    const int r = r0 + t;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (r < n_rows && r % c.a.T < c.s.n) {
      x = __ldg(reinterpret_cast<const uint4*>(q + static_cast<long long>(r) * DK) + 2 * u);
      y = __ldg(reinterpret_cast<const uint4*>(q + static_cast<long long>(r) * DK) + 2 * u + 1);
    }
    permute32<KB>(x, y);
    st_shared(dst + chunk_at(t, 2 * u), x);
    st_shared(dst + chunk_at(t, 2 * u + 1), y);
  }
}

// An mbarrier wait that gives up after a second and tells the whole CTA.
struct Waiter {
  volatile int* fail;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (!*fail && ptx::mbar_wait_bounded(bar, parity, kWaitNs)) return true;
    *fail = 1;
    return false;
  }
};

// The producers' loop: tiles t.begin .. t.end of the CTA into stages 0, 1, 0, ...
template <int KB, int VB, int DK, int MT>
__device__ __forceinline__ void produce(const Ctx& c, const Tiles& t, int r0, int n_rows, int tid, uint32_t base,
                                        uint32_t bars, const Waiter& wait) {
  using Lay = Layout<DK, MT>;
  constexpr bool kPacked = KB != 16;
  constexpr int NK = kPacked ? KeyUnits<KB == 16 ? 8 : KB, DK>::kTokens * (KB == 8 ? 2 : 1) : 1;
  constexpr int NV = kPacked ? 2 * VB : 1;
  const int lane = tid & 31;
  const int n = t.end - t.begin;
  uint32_t wk[NK], wv[NV];
  auto prefetch = [&](int it) {
    if constexpr (kPacked) {
      if (it < n && t.begin + it < t.nq) {
        const int p0 = (t.begin + it) * kTile;
        load_key_codes<KB, DK>(c, p0, tid, wk);
        load_value_codes<VB>(c, p0, tid, wv);
      }
    }
  };
  auto meta = [&](int it) {
    if constexpr (kPacked)
      if (it < n && t.begin + it < t.nq)
        fetch_meta<DK>(c, (t.begin + it) * kTile, tid, base + Lay::kMeta + (it & 1) * kMetaStage);
  };
  auto arrive = [&](int bar) {
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * bar);
  };
  // A wait that runs out ends a warp's work, not its loop: the producers' barrier counts every warp.
  bool live = true;
  meta(0);
  prefetch(0);
  for (int i = 0; i < MT; ++i)
    copy_queries<KB, DK>(c, r0 + i * kTile, n_rows, tid, base + Lay::kQ + i * Lay::KH * kHalf);
  for (int it = 0; it < n; ++it) {
    const int tile = t.begin + it, st = it & 1, ph = ((it >> 1) & 1) ^ 1;
    const uint32_t kdst = base + Lay::kK + st * Lay::KH * kHalf, vdst = base + Lay::kV + st * 2 * kHalf;
    const uint32_t mt = base + Lay::kMeta + st * kMetaStage;
    // the tile's (scale, zero) have landed, and everyone is done with the other stage's
    ptx::cp_async_wait_all();
    asm volatile("bar.sync 1, %0;" ::"n"(kProducerThreads) : "memory");
    meta(it + 1);
    live = live && __all_sync(0xffffffffu, wait(bars + 8 * (kKEmpty + st), ph));
    if (!live) continue;
    uint32_t cv[NV];
    if (kPacked && tile < t.nq) {
      const int p0 = tile * kTile;
      if constexpr (kPacked) {
#pragma unroll
        for (int i = 0; i < NV; ++i) cv[i] = wv[i];
        uint32_t ck[NK];
#pragma unroll
        for (int i = 0; i < NK; ++i) ck[i] = wk[i];
        prefetch(it + 1);
        decode_keys<KB, DK>(c, p0, tid, ck, mt, kdst);
      }
    } else {
      const int kind = tile < t.nq + t.nf ? 1 : 2;
      const int e0 = (tile - t.nq - (kind == 2 ? t.nf : 0)) * kTile;
      prefetch(it + 1);
      copy_rows<KB, DK>(c, true, kind, e0, kind == 1 ? t.n_fp16 : t.n_vis, tid, kdst);
    }
    arrive(kKFull + st);
    live = __all_sync(0xffffffffu, wait(bars + 8 * (kVEmpty + st), ph));
    if (!live) continue;
    if (kPacked && tile < t.nq) {
      if constexpr (kPacked) decode_values<VB>(c, tile * kTile, tid, cv, mt + 2048, vdst);
    } else {
      const int kind = tile < t.nq + t.nf ? 1 : 2;
      const int e0 = (tile - t.nq - (kind == 2 ? t.nf : 0)) * kTile;
      copy_rows<VB, kTile>(c, false, kind, e0, kind == 1 ? t.n_fp16 : t.n_vis, tid, vdst);
    }
    arrive(kVFull + st);
  }
  ptx::cp_async_wait_all();
}

template <int DK, int MT>
__device__ __forceinline__ void produce_any(const Ctx& c, const Tiles& t, int r0, int n_rows, int tid, uint32_t base,
                                            uint32_t bars, const Waiter& wait) {
#define KVQ_PRODUCE(K, V) produce<K, V, DK, MT>(c, t, r0, n_rows, tid, base, bars, wait)
  switch (c.d.kb * 32 + c.d.vb) {
    case 2 * 32 + 2: KVQ_PRODUCE(2, 2); break;
    case 2 * 32 + 4: KVQ_PRODUCE(2, 4); break;
    case 2 * 32 + 8: KVQ_PRODUCE(2, 8); break;
    case 4 * 32 + 2: KVQ_PRODUCE(4, 2); break;
    case 4 * 32 + 4: KVQ_PRODUCE(4, 4); break;
    case 4 * 32 + 8: KVQ_PRODUCE(4, 8); break;
    case 8 * 32 + 2: KVQ_PRODUCE(8, 2); break;
    case 8 * 32 + 4: KVQ_PRODUCE(8, 4); break;
    case 8 * 32 + 8: KVQ_PRODUCE(8, 8); break;
    default: KVQ_PRODUCE(16, 16); break;
  }
#undef KVQ_PRODUCE
}

// One thread: S = Q K^T of a (stream, tile), and O (+)= P V.
template <int DK, int MT>
__device__ __forceinline__ void issue_s(uint32_t base, uint32_t tmem, int stream, int st) {
  using Lay = Layout<DK, MT>;
  const uint32_t q = base + Lay::kQ + (MT == 2 ? stream : 0) * Lay::KH * kHalf;
  const uint32_t k = base + Lay::kK + st * Lay::KH * kHalf;
#pragma unroll
  for (int s = 0; s < DK / 16; ++s) {
    const uint32_t off = (s >> 2) * kHalf + (s & 3) * 32;
    mma_ss(tmem + stream * kTile, desc_sw128(q + off, 16), desc_sw128(k + off, 16), kIdesc, s > 0);
  }
}
template <int DK, int MT>
__device__ __forceinline__ void issue_pv(uint32_t base, uint32_t tmem, int stream, int st, bool acc) {
  const uint32_t v = base + Layout<DK, MT>::kV + st * 2 * kHalf;
#pragma unroll
  for (int s = 0; s < kTile / 16; ++s)
    mma_ts(tmem + 2 * kTile + stream * kTile, tmem + stream * kTile + 8 * s, desc_sw128(v + s * 2048, kHalf), kIdescPV,
           acc || s > 0);
}

template <int DK, int MT>
__device__ __forceinline__ void run_mma(uint32_t base, uint32_t bars, uint32_t tmem, int n, const Waiter& wait) {
  auto bar = [&](int i) { return bars + 8 * i; };
  if constexpr (MT == 2) {
    // both streams use every tile
    bool ok = wait(bar(kKFull), 0);
    if (ok) {
      fence_after();
      issue_s<DK, MT>(base, tmem, 0, 0);
      commit(bar(kSFull));
      issue_s<DK, MT>(base, tmem, 1, 0);
      commit(bar(kSFull + 1));
      commit(bar(kKEmpty));
    }
    for (int it = 0; ok && it < n; ++it) {
      const int st = it & 1, ph = (it >> 1) & 1, st1 = (it + 1) & 1, ph1 = ((it + 1) >> 1) & 1;
      ok = wait(bar(kVFull + st), ph) && wait(bar(kPFull), it & 1);
      if (!ok) break;
      fence_after();
      issue_pv<DK, MT>(base, tmem, 0, st, it > 0);
      if (it + 1 < n) {
        ok = wait(bar(kKFull + st1), ph1);
        if (!ok) break;
        fence_after();
        issue_s<DK, MT>(base, tmem, 0, st1);
        commit(bar(kSFull));
      }
      ok = wait(bar(kPFull + 1), it & 1);
      if (!ok) break;
      fence_after();
      issue_pv<DK, MT>(base, tmem, 1, st, it > 0);
      commit(bar(kVEmpty + st));
      if (it + 1 < n) {
        issue_s<DK, MT>(base, tmem, 1, st1);
        commit(bar(kSFull + 1));
        commit(bar(kKEmpty + st1));
      }
    }
  } else {
    // the streams take alternate tiles
    bool ok = true;
    auto score = [&](int u) {
      const int st = u & 1;
      ok = ok && wait(bar(kKFull + st), (u >> 1) & 1);
      if (!ok) return;
      fence_after();
      issue_s<DK, MT>(base, tmem, st, st);
      commit(bar(kSFull + st));
      commit(bar(kKEmpty + st));
    };
    score(0);
    if (n > 1) score(1);
    for (int u = 0; ok && u < n; ++u) {
      const int st = u & 1, ph = (u >> 1) & 1;
      ok = wait(bar(kVFull + st), ph) && wait(bar(kPFull + st), ph);
      if (!ok) break;
      fence_after();
      issue_pv<DK, MT>(base, tmem, st, st, u > 1);
      commit(bar(kVEmpty + st));
      if (u + 2 < n) score(u + 2);
    }
  }
  commit(bar(kODone));
  // everything issued has to end before the CTA frees its TMEM, also after a failed wait
  if (!ptx::mbar_wait_bounded(bar(kODone), 0, kWaitNs)) *wait.fail = 1;
}

// The lowest x bits of a word (all for x >= 32, none for x <= 0).
__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u; }

// Undo the values' channel order: y[channel] = x[position] within 32 columns.
template <int VB>
__device__ __forceinline__ int column_of(int ch) {
  if constexpr (VB == 16) return ch;
  constexpr int P = VB == 16 ? 1 : 32 / VB, H = P / 2;
  const int q = ch % P;
  return ch - q + (q < H ? 2 * q : 2 * (q - H) + 1);
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
chunk_mma_kernel(const __grid_constant__ Dims d, const __grid_constant__ CacheBufs cb,
                 const __grid_constant__ ChunkArgs a) {
  using Lay = Layout<DK, MT>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  __shared__ uint32_t sm_tmem;
  __shared__ int sm_fail;

  const int split = blockIdx.x % a.splits, rb = blockIdx.x / a.splits, h = blockIdx.y, b = blockIdx.z;
  const int bh = b * d.Hkv + h;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const SeqNew s = seq_new(a.seq, b, d.log_retain);
  const int n_rows = d.n_rep * a.T, r0 = rb * MT * kTile;

  // new tokens that a row of this block may see; a block of which no row is valid ends here
  Tiles t;
  {
    const int r1 = min(r0 + MT * kTile, n_rows) - 1;
    const int t0 = r0 % a.T, t1 = r1 % a.T;
    const bool wraps = r1 / a.T != r0 / a.T;          // the block ends one head's rows and begins another's
    if (s.n == 0 || (!wraps && t0 >= s.n)) return;
    t.n_vis = a.mask || wraps ? s.n : min(s.n, t1 + 1);
    t.n_fp16 = s.n_ret + s.L - s.Q;
    t.nq = (s.Q + kTile - 1) / kTile;
    t.nf = (t.n_fp16 + kTile - 1) / kTile;
    const int all = t.nq + t.nf + (t.n_vis + kTile - 1) / kTile;
    t.begin = static_cast<int>(static_cast<long long>(split) * all / a.splits);
    t.end = static_cast<int>(static_cast<long long>(split + 1) * all / a.splits);
  }
  const int n = t.end - t.begin;

  const uint32_t bars = base + Lay::kBars;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars + 8 * (kKFull + i), kProducerWarps);
      ptx::mbar_init(bars + 8 * (kKEmpty + i), 1);
      ptx::mbar_init(bars + 8 * (kVFull + i), kProducerWarps);
      ptx::mbar_init(bars + 8 * (kVEmpty + i), 1);
      ptx::mbar_init(bars + 8 * (kSFull + i), 1);
      ptx::mbar_init(bars + 8 * (kPFull + i), 4);
    }
    ptx::mbar_init(bars + 8 * kODone, 1);
    ptx::fence_barrier_init();
    sm_fail = 0;
  }
  if (warp == kThreads / 32 - 1) tmem_alloc(ptx::smem_addr(&sm_tmem), 512);
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

  if (warp >= 8 && warp < 16) {
    const Ctx c{d, cb, a, s, b, h, bh};
    produce_any<DK, MT>(c, t, r0, n_rows, tid - kSoftmaxThreads, base, bars, wait);
  } else if (warp == 16) {
    if (lane == 0 && n > 0) run_mma<DK, MT>(base, bars, tmem, n, wait);
    __syncwarp();
  } else {
    // ---------------- softmax ----------------
    const uint32_t ts = tmem + stream * kTile + lanes, to = tmem + 2 * kTile + stream * kTile + lanes;
    const int ret_pos = lane < s.n_ret ? retained_position(s.Q, lane) : -1;
    const int mask_words = (a.T + 31) / 32;
    const float alpha = a.score_scale;
    for (int it = MT == 2 ? 0 : stream; it < n; it += MT == 2 ? 1 : 2, ++mine) {
      if (!__all_sync(0xffffffffu, wait(bars + 8 * (kSFull + stream), mine & 1))) break;
      fence_after();
      // columns of the tile this row sees, 32 a word
      const int tile = t.begin + it;
      const int kind = tile < t.nq ? 0 : tile < t.nq + t.nf ? 1 : 2;
      const int e0 = (tile - (kind > 0 ? t.nq : 0) - (kind > 1 ? t.nf : 0)) * kTile;
      const int nv = min(kTile, (kind == 0 ? s.Q : kind == 1 ? t.n_fp16 : t.n_vis) - e0);
      uint32_t see[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) see[c] = below(nv - 32 * c);
      if (kind == 0) {
        // retained tokens are read from the fp16 list
        unsigned hits = __ballot_sync(0xffffffffu, ret_pos >= e0 && ret_pos < e0 + kTile);
        while (hits) {
          const int off = __shfl_sync(0xffffffffu, ret_pos, __ffs(hits) - 1) - e0;
          hits &= hits - 1;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (off >> 5 == c) see[c] &= ~(1u << (off & 31));
        }
      } else if (kind == 2) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j0 = e0 + 32 * c;
          if (!a.mask)
            see[c] &= below(tr + 1 - j0);
          else
            see[c] &= row_ok && j0 < a.T ? a.mask[(static_cast<long long>(b) * a.T + tr) * mask_words + j0 / 32] : 0u;
        }
      }
      const bool full = __all_sync(0xffffffffu, (see[0] & see[1] & see[2] & see[3]) == 0xffffffffu);

      // ---- the row's maximum ----
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        tmem_ld32(ts + 32 * c, x);
        tmem_wait_ld();
        if (full) {
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(x[i]));
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            mx = fmaxf(mx, (see[c] >> i) & 1u ? __uint_as_float(x[i]) : -INFINITY);
        }
      }
      const float m_new = mx * alpha;
      if (__any_sync(0xffffffffu, m_new > m_ref + kLazy)) {
        const float m2 = fmaxf(m_ref, m_new);
        const float f = m2 == -INFINITY ? 1.0f : ptx::ex2(m_ref - m2);
        m_ref = m2;
        l *= f;
        // S of this tile is committed behind the stream's last P V, so O is complete
        if (mine > 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32(to + 32 * c, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
            tmem_st32(to + 32 * c, x);
          }
        }
      }
      // ---- the weights, over the scores' columns ----
      const float off = kBias - (m_ref == -INFINITY ? 0.0f : m_ref);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32], p[16];
        tmem_ld32(ts + 32 * c, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float s0 = __uint_as_float(x[i]), s1 = __uint_as_float(x[i + 1]);
          if (!full) {
            s0 = (see[c] >> i) & 1u ? s0 : -INFINITY;
            s1 = (see[c] >> (i + 1)) & 1u ? s1 : -INFINITY;
          }
          const float p0 = ptx::ex2(fmaf(s0, alpha, off)), p1 = ptx::ex2(fmaf(s1, alpha, off));
          l += p0 + p1;
          p[i / 2] = ptx::h2_as_u32(__floats2half2_rn(p0, p1));
        }
        tmem_st16(ts + 16 * c, p);
      }
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (kPFull + stream));
    }
    if (n > 0 && !wait(bars + 8 * kODone, 0)) sm_fail = 1;
    fence_after();
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
      asm volatile("bar.sync 2, %0;" ::"n"(kSoftmaxThreads) : "memory");
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
  if (warp == kThreads / 32 - 1) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

template <int DK, int MT>
cudaError_t launch(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(chunk_mma_kernel<DK, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Layout<DK, MT>::kBytes);
  if (e != cudaSuccess) return e;
  const int row_blocks = (d.n_rep * a.T + MT * kTile - 1) / (MT * kTile);
  chunk_mma_kernel<DK, MT><<<dim3(a.splits * row_blocks, d.Hkv, d.B), kThreads, Layout<DK, MT>::kBytes, s>>>(d, c, a);
  return cudaGetLastError();
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
  const int mt = d.n_rep * T > kTile ? 2 : 1;
  const long long units = static_cast<long long>(d.B) * d.Hkv * ((d.n_rep * T + mt * kTile - 1) / (mt * kTile));
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
  const bool wide = d.n_rep * a.T > kTile;
  switch (d.dk) {
    case 32: return wide ? launch<32, 2>(d, c, a, s) : launch<32, 1>(d, c, a, s);
    case 64: return wide ? launch<64, 2>(d, c, a, s) : launch<64, 1>(d, c, a, s);
    default: return wide ? launch<128, 2>(d, c, a, s) : launch<128, 1>(d, c, a, s);
  }
}

}  // namespace kvq
