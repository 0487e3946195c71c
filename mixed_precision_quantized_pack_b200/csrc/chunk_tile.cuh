// The token side of the tensor-core chunk kernels: tiles of 128 tokens of a packed cache, its
// fp16 list and the new tokens, decoded to fp16 in shared memory by eight producer warps.
//
// A tile is written in the 128-byte swizzle that tcgen05.mma reads, a token per 128-byte row of
// 64 channels: keys are K-major and values MN-major operands without any transposition.  The
// packed tiles (codes and (scale, zero) blocks, whole key groups) come through a ring of stages
// in shared memory, filled by bulk copies: nothing a producer thread has asked for itself is
// under way when it publishes its part of a tile, because the proxy fence in front of that waits
// for the thread's own outstanding loads (codes prefetched into registers cost 4700 cycles a tile
// that way; the ring takes about a third).
//
// A code pair masked out of a packed word sits in the two halves of a register, so decoding
// yields channels (i, i + 16 / bits) next to each other.  The channel order of a dot product is
// free: queries and fp16 rows are written in that order too, and the order of the value channels
// is undone where outputs are stored.  Per pair: one LOP3 (1024 + code), one exact operation that
// removes the 1024 and the field's offset, one fused multiply-add that rounds code * s + z to
// fp16 once.  A prefix may end inside its last tile: the rest of that stage holds codes of an older
// tile, or whatever shared memory held.  Its scores are masked before use and its weights are 0; its
// values are finite because the values' (scale, zero) area is cleared in the beginning (clear_ring)
// and holds nothing but finite pairs afterwards.
#pragma once

#include <algorithm>
#include <type_traits>

#include "../../include/kvq.h"
#include "ptx.cuh"
#include "seq_ops.cuh"

namespace kvq {
namespace chunk {

constexpr int kTile = 128;                    // tokens per tile; also the value channels
constexpr int kHalf = kTile * 128;            // bytes of 128 rows of 64 fp16 channels
constexpr int kProducers = 256;               // threads that decode a tile
constexpr int kMaxRing = 4;                   // stages of the packed ring, at most
constexpr int kMetaBytes = 4096;              // (scale, zero) of a tile: keys 2 KB, values 2 KB
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : KVQ_R4(r, 0), KVQ_R4(r, 4), KVQ_R4(r, 8), KVQ_R4(r, 12)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : KVQ_R4(r, 0), KVQ_R4(r, 4), KVQ_R4(r, 8), KVQ_R4(r, 12), KVQ_R4(r, 16), KVQ_R4(r, 20), KVQ_R4(r, 24),
        KVQ_R4(r, 28), KVQ_R4(r, 32), KVQ_R4(r, 36), KVQ_R4(r, 40), KVQ_R4(r, 44), KVQ_R4(r, 48), KVQ_R4(r, 52),
        KVQ_R4(r, 56), KVQ_R4(r, 60)
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
// One lane of a converged warp, the same one every time.  MMAs, commits and bulk copies take uniform
// registers: under this predicate their operands are computed once per warp, while under a
// predicate on the thread index each is moved over lane by lane (about 100 cycles an operation).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Whether a phase has completed (try_wait may suspend the thread; this does not).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major (Q, K): 8-row groups 1024 bytes
// apart.  MN-major (V): 8-token groups 1024 bytes apart, 64-channel halves kHalf apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | static_cast<uint64_t>(lbo >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// f16 x f16 -> f32, 128 rows, n columns; A or B MN-major.
__host__ __device__ constexpr uint32_t instr_desc(int n, bool a_mn, bool b_mn) {
  return 1u << 4 | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | static_cast<uint32_t>(n / 8) << 17 |
         static_cast<uint32_t>(kTile / 16) << 24;
}

// The lowest x bits of a word (all for x >= 32, none for x <= 0).
__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u; }

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

// 16-byte chunk j (8 channels) of row t of ROWS 128-byte rows in the 128-byte swizzle; every 64
// channels a block of rows of its own.
template <int ROWS = kTile>
__device__ __forceinline__ uint32_t chunk_at(int t, int j) {
  return (j >> 3) * (ROWS * 128) + t * 128 + (((j & 7) ^ (t & 7)) << 4);
}
__device__ __forceinline__ void st_shared(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 ld_shared64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
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

// The token tiles of a CTA: quantized, fp16 list (retained, window), new tokens, in this order.
struct Tiles {
  int nq, nf, begin, end;     // quantized tiles, fp16-list tiles; the CTA's range of all tiles
  int n_fp16, n_vis;          // entries of the fp16 list; new tokens that some row of the CTA may see
};

// Tiles of a block of rows r0 .. r1 (inclusive) of the n_rep * T rows; false when none of them is
// valid.
__device__ __forceinline__ bool block_tiles(const ChunkArgs& a, const SeqNew& s, int r0, int r1, int split, Tiles& t) {
  const int t0 = r0 % a.T, t1 = r1 % a.T;
  const bool wraps = r1 / a.T != r0 / a.T;            // the block ends one head's rows and begins another's
  if (s.n == 0 || (!wraps && t0 >= s.n)) return false;
  t.n_vis = a.mask || wraps ? s.n : min(s.n, t1 + 1);
  t.n_fp16 = s.n_ret + s.L - s.Q;
  t.nq = (s.Q + kTile - 1) / kTile;
  t.nf = (t.n_fp16 + kTile - 1) / kTile;
  const int all = t.nq + t.nf + (t.n_vis + kTile - 1) / kTile;
  t.begin = static_cast<int>(static_cast<long long>(split) * all / a.splits);
  t.end = static_cast<int>(static_cast<long long>(split + 1) * all / a.splits);
  return true;
}

// Position of word w of a key row of W words in its group's (scale, zero) block, and the word at a
// position.
template <int W>
__host__ __device__ constexpr int block_pos(int w) { return key_block_pos(W, w); }
template <int W>
__host__ __device__ constexpr int block_word(int p) { return W % 4 == 0 ? p % 4 * (W / 4) + p / 4 : p; }

// Where chunk j (8 channels) of a key or query row is written.
template <int KB, int DK>
__host__ __device__ constexpr int key_chunk(int j) {
  return KB == 4 ? block_pos<DK / 8>(j) : KB == 2 ? block_pos<DK / 16>(j / 2) * 2 + j % 2 : j;
}

// A thread's share of a tile's packed keys: one unit of the row (a chunk of 8 channels, or 16 at
// 2 bits), tokens sub, sub + kStep, ...  At 4 and 2 bits consecutive threads take the words in the
// order of the (scale, zero) blocks and write them in that order too: threads then read
// neighbouring blocks and write neighbouring chunks, and the order of the channels of a dot
// product is free (key_chunk() gives it to the queries and fp16 rows).
template <int KB, int DK>
struct KeyUnits {
  static __host__ __device__ constexpr int unit(int e) { return KB == 8 ? e : block_word<DK * KB / 32>(e); }
  static constexpr int kPerRow = KB == 2 ? DK / 16 : DK / 8;
  static constexpr int kWords = KB == 8 ? 2 : 1;
  static constexpr int kStep = kProducers / kPerRow;
  static constexpr int kTokens = kTile / kStep;
  static_assert(kStep <= kTile, "every thread has tokens");
};

// What the producers of a CTA share.
struct Ctx {
  const Dims& d;
  const CacheBufs& cb;
  const ChunkArgs& a;
  const SeqNew& s;
  int b, h, bh;
  int lgk, lgv, lnvg;         // log2 of the group sizes and of the value groups per token
  uint32_t ring, pages;       // shared memory: the packed ring, the pages of the next tile to copy (16 bytes)
  int stages;                 // of the ring
};

// A stage of the packed ring: key codes, value codes, key (scale, zero) blocks, value (scale, zero).
__host__ __device__ constexpr int ring_stage_bytes(int kb, int vb, int dk) {
  return kb == 16 ? 0 : kTile * (dk * kb + kTile * vb) / 8 + kMetaBytes;
}

// The thread's codes of the key tile in the ring stage `src` to fp16 rows at `dst`.
template <int KB, int DK>
__device__ __forceinline__ void decode_keys(const Ctx& c, int tid, uint32_t src, uint32_t meta, uint32_t dst) {
  using U = KeyUnits<KB, DK>;
  constexpr int P = 32 / KB, W = DK / P, kRow = DK * KB / 8;
  const int u = tid % U::kPerRow, sub = tid / U::kPerRow;
  // (scale, zero) pairs of the unit, reloaded where the next group may begin
  constexpr int R = U::kWords * P / 2;
  uint32_t sc[R], zr[R];
  uint32_t at[U::kWords];
#pragma unroll
  for (int k = 0; k < U::kWords; ++k) at[k] = meta + (KB == 8 ? block_pos<W>(u * U::kWords + k) : u) * (4 * P);
  src += sub * kRow + U::unit(u) * (4 * U::kWords);
  // all loads first: stores and loads of shared memory keep their order, so a load behind a store
  // would wait for it
  uint32_t w[U::kTokens * U::kWords];
#pragma unroll
  for (int i = 0; i < U::kTokens; ++i) {
    if constexpr (KB == 8) {
      const uint2 x = ld_shared64(src + i * (U::kStep * kRow));
      w[2 * i] = x.x;
      w[2 * i + 1] = x.y;
    } else {
      w[i] = ld_shared32(src + i * (U::kStep * kRow));
    }
  }
#pragma unroll
  for (int i = 0; i < U::kTokens; ++i) {
    const int t = sub + i * U::kStep;
    if (i == 0 || U::kStep > 32 || (i * U::kStep % 32 == 0 && ((i * U::kStep) & (c.d.gk - 1)) == 0)) {
      const uint32_t g = (t >> c.lgk) * (DK * 4);
#pragma unroll
      for (int k = 0; k < U::kWords; ++k) {
        if constexpr (KB == 4) {
          // 32-byte blocks, a 16-byte half at a time: every other group of four threads takes the zeros
          // first, so that eight threads read eight different bank groups
          const bool swap = (u >> 2) & 1;
          const uint4 p = ld_shared(at[k] + g + (swap ? 16 : 0)), q = ld_shared(at[k] + g + (swap ? 0 : 16));
          sc[0] = swap ? q.x : p.x;
          sc[1] = swap ? q.y : p.y;
          sc[2] = swap ? q.z : p.z;
          sc[3] = swap ? q.w : p.w;
          zr[0] = swap ? p.x : q.x;
          zr[1] = swap ? p.y : q.y;
          zr[2] = swap ? p.z : q.z;
          zr[3] = swap ? p.w : q.w;
        } else if constexpr (KB == 2) {
          // 64-byte blocks (pairs 0-3 and 4-7 of the scales, then of the zeros): threads with u & 4
          // take the upper pairs first, which halves the bank conflicts of these loads and leaves the
          // stores below none (8 tokens, 16 x 16k, K2V2: 327 -> 214 us with one load per group)
          const int f1 = (u >> 2) & 1;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 p = ld_shared(at[k] + g + (e ^ f1) * 16), q = ld_shared(at[k] + g + ((e ^ f1) + 2) * 16);
            sc[4 * e] = p.x;
            sc[4 * e + 1] = p.y;
            sc[4 * e + 2] = p.z;
            sc[4 * e + 3] = p.w;
            zr[4 * e] = q.x;
            zr[4 * e + 1] = q.y;
            zr[4 * e + 2] = q.z;
            zr[4 * e + 3] = q.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < P; e += 4) {       // P registers: P / 2 scale pairs, then P / 2 zero pairs
            const uint4 m = ld_shared(at[k] + g + 4 * e);
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
      // the pairs 4-7 lie eight bits above 0-3
      const uint32_t x = (u & 4) ? w[i] >> 8 : w[i], y = (u & 4) ? w[i] : w[i] >> 8;
      o[0] = decode_pair<2, 0>(x, sc[0], zr[0]);
      o[1] = decode_pair<2, 1>(x, sc[1], zr[1]);
      o[2] = decode_pair<2, 2>(x, sc[2], zr[2]);
      o[3] = decode_pair<2, 3>(x, sc[3], zr[3]);
      o[4] = decode_pair<2, 0>(y, sc[4], zr[4]);
      o[5] = decode_pair<2, 1>(y, sc[5], zr[5]);
      o[6] = decode_pair<2, 2>(y, sc[6], zr[6]);
      o[7] = decode_pair<2, 3>(y, sc[7], zr[7]);
    }
#pragma unroll
    for (int e = 0; e < R; e += 4)
      st_shared(dst + chunk_at(t, u * (R / 4) + (KB == 2 ? e / 4 ^ ((u >> 2) & 1) : e / 4)), make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
  }
}

// Values: a thread decodes 64 channels of a token, in two blocks.  Threads of a row's second half
// take their blocks in the opposite order, so that the eight threads of a store phase write eight
// different bank groups.
template <int VB>
__device__ __forceinline__ void decode_values(const Ctx& c, int tid, uint32_t src, uint32_t meta, uint32_t dst) {
  constexpr int kPerRow = kProducers / kTile, kChannels = kTile / kPerRow;       // threads a token, channels a thread
  constexpr int C = kChannels / 16, B = kChannels / 2 * VB / 32;         // chunks and words of a block
  const int e = tid % kPerRow, t = tid / kPerRow, flip = e >= kPerRow / 2;
  const uint32_t row = meta + ((t << c.lnvg) * 4);
  const uint32_t to = dst + t * 128 + (e * kChannels >= 64 ? kHalf : 0);
  src += t * (16 * VB) + e * (8 * B);
  uint32_t wp[2][B], sz[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if constexpr (B == 1) {
      wp[p][0] = ld_shared32(src + (p ^ flip) * 4);
    } else if constexpr (B == 2) {
      const uint2 x = ld_shared64(src + (p ^ flip) * 8);
      wp[p][0] = x.x;
      wp[p][1] = x.y;
    } else {
#pragma unroll
      for (int k = 0; k < B; k += 4) {
        const uint4 x = ld_shared(src + (p ^ flip) * (4 * B) + 4 * k);
        wp[p][k] = x.x;
        wp[p][k + 1] = x.y;
        wp[p][k + 2] = x.z;
        wp[p][k + 3] = x.w;
      }
    }
    // groups hold at least 32 channels: one (scale, zero) a block
    sz[p] = ld_shared32(row + (8 * (e * (kChannels / 8) + (p ^ flip) * C) >> c.lgv) * 4);
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int j0 = e * (kChannels / 8) + (p ^ flip) * C;             // first chunk of the block
    const uint32_t(&w)[B] = wp[p];
    const uint32_t s = ptx::prmt(sz[p], sz[p], 0x1010), z = ptx::prmt(sz[p], sz[p], 0x3232);
    const uint32_t x7 = (j0 & 7) ^ (t & 7);                          // C is a power of two and divides j0
#pragma unroll
    for (int k = 0; k < C; ++k) {
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
      st_shared(to + ((x7 ^ k) << 4), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

// fp16 rows of the list (kind 1) or of the new tokens (kind 2) to a tile; entries from `n` on are zero.
// WIDTH channels a row; the channel order is that of BITS-bit codes.
template <int BITS, int WIDTH>
__device__ __forceinline__ void copy_rows(const Ctx& c, bool keys, int kind, int e0, int n, int tid, uint32_t dst) {
  constexpr int per_row = WIDTH / 16, step = kProducers / per_row, tokens = kTile / step;
  static_assert(step <= kTile, "every thread has rows");
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
    const int j0 = keys ? key_chunk<BITS, WIDTH>(2 * u) : 2 * u, j1 = keys ? key_chunk<BITS, WIDTH>(2 * u + 1) : 2 * u + 1;
    st_shared(dst + chunk_at(t, j0), x[i]);
    st_shared(dst + chunk_at(t, j1), y[i]);
  }
}

// ROWS query rows from r0 of the kv head's block (rows of T tokens per head; those behind the
// sequence's new tokens are zero), in the keys' channel order.
template <int KB, int DK, int ROWS>
__device__ __forceinline__ void copy_queries(const Ctx& c, int r0, int n_rows, int tid, uint32_t dst) {
  constexpr int per_row = DK / 16, step = kProducers / per_row;
  const int u = tid % per_row, sub = tid / per_row;
  const __half* q = c.a.q + static_cast<long long>(c.bh) * n_rows * DK;
  for (int t = sub; t < ROWS; t += step) {
    const int r = r0 + t;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (r < n_rows && r % c.a.T < c.s.n) {
      x = __ldg(reinterpret_cast<const uint4*>(q + static_cast<long long>(r) * DK) + 2 * u);
      y = __ldg(reinterpret_cast<const uint4*>(q + static_cast<long long>(r) * DK) + 2 * u + 1);
    }
    permute32<KB>(x, y);
    st_shared(dst + chunk_at<ROWS>(t, key_chunk<KB, DK>(2 * u)), x);
    st_shared(dst + chunk_at<ROWS>(t, key_chunk<KB, DK>(2 * u + 1)), y);
  }
}

// An mbarrier wait that gives up after a second and tells the whole CTA.  The waits hand tiles from
// role to role several times a microsecond, so they take the plain try_wait: with a suspend-time
// hint a waiting warp sleeps and wakes up late.
struct Waiter {
  volatile int* fail;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    for (;;) {
#pragma unroll 1
      for (int i = 0; i < 16; ++i)
        if (ptx::mbar_try_wait(bar, parity)) return true;
      if (*fail || ptx::globaltimer() - t0 > kWaitNs) break;
    }
    *fail = 1;
    return false;
  }
};

// Barriers between producers and the MMA thread (pairs: one per stage), and of the packed ring.
enum TokenBars { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kRingFull = 8, kRingEmpty = 12, kTokenBars = 16 };

// The stages of a packed ring that fit beside `used` bytes of shared memory.
constexpr int kMaxSmem = 232448 - 64;           // dynamic, beside the kernels' few static bytes
inline int ring_stages(const Dims& d, int used) {
  const int bytes = ring_stage_bytes(d.kb, d.vb, d.dk);
  return bytes == 0 ? 0 : std::min(kMaxRing, (kMaxSmem - used) / bytes);
}

// Zeros in the value (scale, zero) of every ring stage: a prefix's last tile may be shorter than the
// stage, and the values behind it, whose weights are 0, have to be finite.  By all threads of the
// CTA, before the barrier in front of the roles.
__device__ __forceinline__ void clear_ring(const Dims& d, uint32_t ring, int stages, int tid, int threads) {
  const int bytes = ring_stage_bytes(d.kb, d.vb, d.dk);
  for (int i = tid; i < stages * (kMetaBytes / 32); i += threads) {
    const int st = i / (kMetaBytes / 32), e = i % (kMetaBytes / 32);
    st_shared(ring + st * bytes + bytes - kMetaBytes / 2 + e * 16, make_uint4(0, 0, 0, 0));
  }
  ptx::fence_proxy_async_smem();
}

// Arrivals a phase: `producers` warps that write keys, as many that write values, `readers` warps of
// the packed ring, `users` MMA streams of a tile.
__device__ __forceinline__ void init_token_bars(uint32_t bars, int producers, int readers, int users) {
  for (int i = 0; i < 2; ++i) {
    ptx::mbar_init(bars + 8 * (kKFull + i), producers);
    ptx::mbar_init(bars + 8 * (kKEmpty + i), users);
    ptx::mbar_init(bars + 8 * (kVFull + i), producers);
    ptx::mbar_init(bars + 8 * (kVEmpty + i), users);
  }
  for (int i = 0; i < kMaxRing; ++i) {
    ptx::mbar_init(bars + 8 * (kRingFull + i), 1);
    ptx::mbar_init(bars + 8 * (kRingEmpty + i), readers);
  }
}

// One warp (converged) copies packed tile `tile` into ring stage `slot`: an unpaged sequence's tile is
// four contiguous runs, a paged one's four per key group.
template <int KB, int VB, int DK>
__device__ __forceinline__ void copy_tile(const Ctx& c, int tile, int slot, int lane, uint32_t bars) {
  const Dims& d = c.d;
  constexpr int kRowK = DK * KB / 8, kRowV = kTile * VB / 8;
  const int g0 = (tile * kTile) >> c.lgk, groups = min(kTile >> c.lgk, (c.s.Q >> c.lgk) - g0);
  const uint32_t bar = bars + 8 * (kRingFull + slot);
  const uint32_t dst = c.ring + slot * ring_stage_bytes(KB, VB, DK);
  const uint32_t kbytes = d.gk * kRowK, vbytes = d.gk * kRowV, zbytes = (d.gk << c.lnvg) * 4;
  const char* kc = reinterpret_cast<const char*>(c.cb.kcode);
  const char* vc = reinterpret_cast<const char*>(c.cb.vcode);
  const char* km = reinterpret_cast<const char*>(c.cb.ksz);
  const char* vm = reinterpret_cast<const char*>(c.cb.vsz);
  auto copy = [&](long long gidx, int i, uint32_t n) {       // n groups from gidx on, to place i of the stage
    ptx::bulk_g2s(dst + i * kbytes, kc + gidx * kbytes, n * kbytes, bar);
    ptx::bulk_g2s(dst + kTile * (kRowK + kRowV) + i * (DK * 4), km + gidx * (DK * 4), n * (DK * 4), bar);
    ptx::bulk_g2s(dst + kTile * kRowK + i * vbytes, vc + gidx * vbytes, n * vbytes, bar);
    ptx::bulk_g2s(dst + kTile * (kRowK + kRowV) + kMetaBytes / 2 + i * zbytes, vm + gidx * zbytes, n * zbytes, bar);
  };
  if (d.paged) ptx::cp_async_wait_all();          // the tile's pages
  __syncwarp();
  if (elect_one()) {
    ptx::fence_proxy_async_smem();                // the stage's last readers are behind the ring's barrier
    ptx::mbar_arrive_expect_tx(bar, groups * (kbytes + vbytes + DK * 4 + zbytes));
    if (d.paged) {
      for (int i = 0; i < groups; ++i) {
        long long gidx = static_cast<long long>(static_cast<int>(ld_shared32(c.pages + 4 * i))) * d.Hkv + c.h;
        // (bounds-check builds) a group outside the buffers is replaced by group 0
        if (!KVQ_IN_BOUNDS(d, kSiteChunkGroup, gidx, quant_groups(d))) gidx = 0;
        copy(gidx, i, 1);
      }
    } else {
      long long gidx = static_cast<long long>(c.bh) * d.max_groups + g0;
      if (!KVQ_RANGE_IN_BOUNDS(d, kSiteChunkGroup, gidx, groups, quant_groups(d))) gidx = 0;
      copy(gidx, 0, groups);
    }
  }
  __syncwarp();
  // the pages of the next tile, while there is one
  const int g1 = g0 + (kTile >> c.lgk) + lane;
  if (d.paged && lane < (kTile >> c.lgk) && (g1 << c.lgk) < c.s.Q && KVQ_IN_BOUNDS(d, kSiteChunkTable, g1, d.max_groups))
    ptx::cp_async_4(c.pages + 4 * lane, c.cb.table + c.b * d.max_groups + g1);
}

// The copying warp's side of the packed ring.
template <int KB, int VB, int DK>
struct Copier {
  int packed = 0, copied = 0;                   // the CTA's packed tiles, and those asked for
  // the first tiles, a ring's length of them
  __device__ __forceinline__ void start(const Ctx& c, const Tiles& t, int n, int lane, uint32_t bars) {
    packed = n;
    if (packed <= 0) return;
    if (c.d.paged) {
      const int g = ((t.begin * kTile) >> c.lgk) + lane;
      if (lane < (kTile >> c.lgk) && (g << c.lgk) < c.s.Q && KVQ_IN_BOUNDS(c.d, kSiteChunkTable, g, c.d.max_groups))
        ptx::cp_async_4(c.pages + 4 * lane, c.cb.table + c.b * c.d.max_groups + g);
    }
    for (; copied < c.stages && copied < packed; ++copied) copy_tile<KB, VB, DK>(c, t.begin + copied, copied, lane, bars);
  }
  // the next tile, into the stage of the one a ring's length before it, once every producer has read that
  __device__ __forceinline__ bool next(const Ctx& c, const Tiles& t, int lane, uint32_t bars, const Waiter& wait) {
    if (copied >= packed) return true;
    const int slot = copied % c.stages;
    if (!__all_sync(0xffffffffu, wait(bars + 8 * (kRingEmpty + slot), (copied / c.stages - 1) & 1))) return false;
    copy_tile<KB, VB, DK>(c, t.begin + copied, slot, lane, bars);
    ++copied;
    return true;
  }
  // no copy may land in shared memory behind the CTA: after a wait that ran out, waits (again with a
  // limit) for the last copies into every stage
  __device__ __forceinline__ void drain(const Ctx& c, int lane, uint32_t bars, bool live) {
    ptx::cp_async_wait_all();
    if (!live && lane < c.stages && lane < copied)
      ptx::mbar_wait_bounded(bars + 8 * (kRingFull + lane), ((copied - lane - 1) / c.stages) & 1, kWaitNs);
  }
};

// The loop of a warp that only copies (the producers' SELF is false then).
template <int KB, int VB, int DK>
__device__ __forceinline__ void copy_tiles(const Ctx& c, const Tiles& t, int lane, uint32_t bars, const Waiter& wait) {
  Copier<KB, VB, DK> copier;
  copier.start(c, t, max(0, min(t.end, t.nq) - t.begin), lane, bars);
  bool live = true;
  while (live && copier.copied < copier.packed) live = copier.next(c, t, lane, bars, wait);
  // the producers' waits tell whether the copies all landed
  copier.drain(c, lane, bars, false);
}

// The loop of the producer threads: tiles t.begin .. t.end of the CTA into stages 0, 1, 0, ... of K and
// V.  SELF: the first warp copies the packed tiles as well.  (Two groups of 256, one for the keys
// and one for the values, gained 6% with 16 queries and lost 11% with 32.)
template <int KB, int VB, int DK, bool SELF>
__device__ __forceinline__ void produce(const Ctx& c, const Tiles& t, int tid, uint32_t kdst0, uint32_t vdst0,
                                        uint32_t bars, const Waiter& wait) {
  constexpr int kKeyStage = (DK > 64 ? DK / 64 : 1) * kHalf;
  constexpr bool kPacked = KB != 16;
  constexpr int kRowK = DK * KB / 8, kRowV = kTile * VB / 8;
  const int lane = tid & 31;
  const int n = t.end - t.begin;
  const int packed = kPacked ? max(0, min(t.end, t.nq) - t.begin) : 0;      // the CTA's first tiles
  auto arrive = [&](int bar) {
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * bar);
  };
  auto ready = [&](int bar, int parity) { return __all_sync(0xffffffffu, wait(bars + 8 * bar, parity)); };
  bool live = true;
  Copier<KB, VB, DK> copier;
  if constexpr (kPacked && SELF)
    if (tid < 32) copier.start(c, t, packed, lane, bars);
  int slot = 0, round = 0;                      // ring stage of tile `it`, and how often the ring went round
  for (int it = 0; live && it < n; ++it) {
    const int tile = t.begin + it, st = it & 1, ph = ((it >> 1) & 1) ^ 1;
    const uint32_t kdst = kdst0 + st * kKeyStage, vdst = vdst0 + st * 2 * kHalf;
    const uint32_t src = c.ring + slot * ring_stage_bytes(KB, VB, DK);
    const int kind = tile < t.nq + t.nf ? 1 : 2, e0 = (tile - t.nq - (kind == 2 ? t.nf : 0)) * kTile;
    const int ne = kind == 1 ? t.n_fp16 : t.n_vis;
    if constexpr (kPacked && SELF)
      if (tid < 32 && it > 0 && !copier.next(c, t, lane, bars, wait)) break;
    if (kPacked && it < packed && !ready(kRingFull + slot, round & 1)) break;
    live = ready(kKEmpty + st, ph);
    if (!live) break;
    if (it < packed) {
      if constexpr (kPacked) decode_keys<KB, DK>(c, tid, src, src + kTile * (kRowK + kRowV), kdst);
    } else {
      copy_rows<KB, DK>(c, true, kind, e0, ne, tid, kdst);
    }
    arrive(kKFull + st);
    live = ready(kVEmpty + st, ph);
    if (!live) break;
    if (it < packed) {
      if constexpr (kPacked) decode_values<VB>(c, tid, src + kTile * kRowK, src + kTile * (kRowK + kRowV) + kMetaBytes / 2, vdst);
    } else {
      copy_rows<VB, kTile>(c, false, kind, e0, ne, tid, vdst);
    }
    arrive(kVFull + st);
    if (kPacked && it < packed) {
      if (lane == 0) mbar_arrive(bars + 8 * (kRingEmpty + slot));
      if (++slot == c.stages) {
        slot = 0;
        ++round;
      }
    }
  }
  if constexpr (kPacked && SELF)
    if (tid < 32) copier.drain(c, lane, bars, *wait.fail == 0);
}

// f with the cache's bit widths as constants.
template <typename F>
__device__ __forceinline__ void with_bits(const Dims& d, const F& f) {
#define KVQ_BITS(K, V) \
  case K * 32 + V:     \
    f(std::integral_constant<int, K>(), std::integral_constant<int, V>()); \
    break;
  switch (d.kb * 32 + d.vb) {
    KVQ_BITS(2, 2)
    KVQ_BITS(2, 4)
    KVQ_BITS(2, 8)
    KVQ_BITS(4, 2)
    KVQ_BITS(4, 4)
    KVQ_BITS(4, 8)
    KVQ_BITS(8, 2)
    KVQ_BITS(8, 4)
    KVQ_BITS(8, 8)
    KVQ_BITS(16, 16)
  }
#undef KVQ_BITS
}

// Undo the values' channel order: y[channel] = x[position] within 32 columns.
template <int VB>
__device__ __forceinline__ int column_of(int ch) {
  if constexpr (VB == 16) return ch;
  constexpr int P = VB == 16 ? 1 : 32 / VB, H = P / 2;
  const int q = ch % P;
  return ch - q + (q < H ? 2 * q : 2 * (q - H) + 1);
}

}  // namespace chunk
}  // namespace kvq
