// Several tokens per sequence appended at once: the state after that many one-token appends.
//
// A sequence of L tokens (Q quantized) that takes n more has Q' = prefix(L + n) quantized
// tokens, so the groups [Q, Q') leave the window.  Their tokens come from the window (positions
// below L) or straight from the new rows, and every group is quantized on its own: one CTA per
// (group, kv head, sequence), plus one CTA per (kv head, sequence) that rebuilds the retained
// list.  A second launch then writes the new tokens that stay in the window; it may overwrite
// window slots whose tokens the first one read, so the two are ordered by the stream.  Without
// a group to quantize only the second launch runs.
//
// Bound: latency for a few accepted tokens, else the bytes of the new rows.  A group is read
// once, into shared memory (rows padded by 16 bytes, so that a column walk touches every bank
// group); its per-channel minima, the packing and the side code all work from there.
#include <algorithm>

#include "quant_math.cuh"
#include "seq_ops.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kPad = 8;   // halves

// Where position p of sequence b, kv head h comes from: a window slot (p < L) or a new row.
struct TokenSource {
  const __half* base;
  bool fresh;   // a new row: keys still unrotated
};
__device__ __forceinline__ TokenSource token_source(const Dims& d, const __half* win, const __half* fresh, int width,
                                                    const int* index, int T, const SeqNew& s, int b, int bh, int p) {
  TokenSource t;
  t.fresh = p >= s.L;
  if (!t.fresh) {
    long long row = static_cast<long long>(bh) * d.cap + p % d.cap;
    if (!KVQ_IN_BOUNDS(d, kSiteTokWin, row, win_rows(d))) row = 0;
    t.base = win + row * width;
  } else {
    const int i = p - s.L;
    int r = index ? index[static_cast<long long>(b) * T + i] : i;
    if (r < 0 || r >= T) r = 0;               // an index outside the chunk reads its first row
    long long row = static_cast<long long>(bh) * T + r;
    if (!KVQ_IN_BOUNDS(d, kSiteTokSrc, row, static_cast<long long>(d.B) * d.Hkv * T)) row = 0;
    t.base = fresh + row * width;
  }
  return t;
}

__device__ __forceinline__ void rotate_smem_row(__half* row, const Dims& d, int lane) {
  float x[8];
#pragma unroll
  for (int m = 0; m < 8; ++m) x[m] = m < d.dk / 32 ? __half2float(row[lane + 32 * m]) : 0.0f;
  rotate_row_warp<8>(x, d.dk / 32, d.rot_signs, d.rot_inv_ck, lane);
#pragma unroll
  for (int m = 0; m < 8; ++m)
    if (m < d.dk / 32) row[lane + 32 * m] = __float2half_rn(x[m]);
}

// Codes of 8 fp16 values, LSB first; prm(j) is (zero, 1 / scale, scale) of value j's group.  The
// reciprocal decides all but quotients next to a half-integer, which take the division.
template <typename P>
__device__ __forceinline__ uint64_t chunk_codes(const uint4& raw, int bits, const P& prm) {
  const __half2* hx = reinterpret_cast<const __half2*>(&raw);
  const uint32_t levels = (1u << bits) - 1u;
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(hx[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
  bool near = false;
  uint64_t codes = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float3 p = prm(j);
    codes |= static_cast<uint64_t>(code_fast_l(x[j], p.x, p.y, levels, near)) << (j * bits);
  }
  if (near) {
    codes = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float3 p = prm(j);
      codes |= static_cast<uint64_t>(code_exact_l(x[j], p.x, p.z, levels)) << (j * bits);
    }
  }
  return codes;
}

// n bits (8, 16, 32 or 64) at bit offset `off`, a multiple of n, of a packed row.
__device__ __forceinline__ void store_codes(uint32_t* row, int off, int n, uint64_t codes) {
  if (n == 64) {
    row[off / 32] = static_cast<uint32_t>(codes);
    row[off / 32 + 1] = static_cast<uint32_t>(codes >> 32);
  } else if (n == 32) {
    row[off / 32] = static_cast<uint32_t>(codes);
  } else if (n == 16) {
    reinterpret_cast<uint16_t*>(row)[off / 16] = static_cast<uint16_t>(codes);
  } else {
    reinterpret_cast<uint8_t*>(row)[off / 8] = static_cast<uint8_t>(codes);
  }
}

// Zeros in the bytes behind the last field of a width map's packed value rows.
__device__ __forceinline__ void zero_tail(const int* cnt, int words, uint32_t* rows, int n, int tid) {
  const int bytes = (cnt[0] * 8 + cnt[1] * 4 + cnt[2] * 2 + cnt[3]) / 8;    // groups of at least 8 channels: whole bytes
  for (int i = tid; i < n * (4 * words - bytes); i += kThreads)
    reinterpret_cast<uint8_t*>(rows + (i / (4 * words - bytes)) * words)[bytes + i % (4 * words - bytes)] = 0;
}

__global__ void __launch_bounds__(kThreads, 4)
append_groups_kernel(Dims d, CacheOut c, SeqChunk w, const __half* __restrict__ k, const __half* __restrict__ v,
                     int T, const int* __restrict__ index, int max_new_groups) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int h = blockIdx.y, b = blockIdx.z, bh = b * d.Hkv + h;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nwarps = kThreads / 32;
  const SeqNew s = seq_new(w, b, d.log_retain);
  const int Q2 = prefix_of(d, s.L + s.n);
  const int ks = d.dk + kPad, vs = d.dv + kPad;     // padded row strides, halves
  const int vk = d.dk / 8, vv = d.dv / 8;
  if (static_cast<int>(blockIdx.x) == max_new_groups) {
    // ---- the retained list of the longer prefix, in place: staged, then written ----
    if (!d.log_retain || Q2 == s.Q) return;
    const int n_new = retained_count(Q2);
    __half* sk = reinterpret_cast<__half*>(smem);
    __half* sv = sk + kMaxRetained * ks;
    for (int i = warp; i < n_new; i += nwarps) {
      const int p = retained_position(Q2, i);
      const __half *pk, *pv;
      bool fresh = false;
      if (p < s.Q) {
        // still retained: its place in the old list is the octave of its old age
        const int at = retained_count(s.Q) - 1 - (31 - __clz(s.Q - p));
        long long row = static_cast<long long>(bh) * kMaxRetained + at;
        if (!KVQ_IN_BOUNDS(d, kSiteRetUpd, row, ret_rows(d))) row = 0;
        pk = c.ret_k + row * d.dk;
        pv = c.ret_v + row * d.dv;
      } else {
        const TokenSource a = token_source(d, c.win_k, k, d.dk, index, T, s, b, bh, p);
        pk = a.base;
        fresh = a.fresh;
        pv = token_source(d, c.win_v, v, d.dv, index, T, s, b, bh, p).base;
      }
      for (int e = lane; e < vk; e += 32)
        reinterpret_cast<uint4*>(sk + i * ks)[e] = reinterpret_cast<const uint4*>(pk)[e];
      for (int e = lane; e < vv; e += 32)
        reinterpret_cast<uint4*>(sv + i * vs)[e] = reinterpret_cast<const uint4*>(pv)[e];
      __syncwarp();
      if (fresh && d.rot) rotate_smem_row(sk + i * ks, d, lane);
    }
    __syncthreads();
    for (int idx = tid; idx < n_new * (vk + vv); idx += kThreads) {
      const int i = idx / (vk + vv), e = idx % (vk + vv);
      const size_t row = static_cast<size_t>(bh) * kMaxRetained + i;
      if (e < vk)
        reinterpret_cast<uint4*>(c.ret_k + row * d.dk)[e] = reinterpret_cast<const uint4*>(sk + i * ks)[e];
      else
        reinterpret_cast<uint4*>(c.ret_v + row * d.dv)[e - vk] = reinterpret_cast<const uint4*>(sv + i * vs)[e - vk];
    }
    return;
  }
  const int g = s.Q / d.gk + blockIdx.x;
  if (g >= Q2 / d.gk) return;
  // shared memory: key rows, value rows, key (scale, zero) and 1 / scale, slabs, side residual sums,
  // side (scale, zero)
  __half* sk = reinterpret_cast<__half*>(smem);
  __half* sv = sk + d.gk * ks;
  float2* kp = reinterpret_cast<float2*>(sv + d.gk * vs);
  float* kr = reinterpret_cast<float*>(kp + d.dk);
  float* vp = kr + d.dk;                            // 4 KB: the slabs' extremes
  float* y = vp + 1024;
  float2* zp = reinterpret_cast<float2*>(y + d.gk * 8);
  const int p0 = g * d.gk;
  // the group's rows, a 16-byte piece per thread and step, eight steps of loads ahead of their stores
  {
    constexpr int kSteps = 8;
    const int total = d.gk * (vk + vv);
    for (int i0 = tid; i0 < total; i0 += kSteps * kThreads) {
      uint4 x[kSteps];
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int i = i0 + j * kThreads, t = i / (vk + vv), e = i % (vk + vv);
        if (i < total)
          x[j] = __ldg(reinterpret_cast<const uint4*>(
                     e < vk ? token_source(d, c.win_k, k, d.dk, index, T, s, b, bh, p0 + t).base
                            : token_source(d, c.win_v, v, d.dv, index, T, s, b, bh, p0 + t).base) + (e < vk ? e : e - vk));
      }
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int i = i0 + j * kThreads, t = i / (vk + vv), e = i % (vk + vv);
        if (i < total) reinterpret_cast<uint4*>(e < vk ? sk + t * ks : sv + t * vs)[e < vk ? e : e - vk] = x[j];
      }
    }
    if (d.rot) {
      __syncthreads();
      for (int t = warp; t < d.gk; t += nwarps)
        if (p0 + t >= s.L) rotate_smem_row(sk + t * ks, d, lane);        // new rows; the window's are rotated
    }
  }
  __syncthreads();
  long long row0 = static_cast<long long>(group_row(d, c.table, b, h, g));
  long long gidx = static_cast<long long>(group_index(d, c.table, b, h, g));
  if (!KVQ_RANGE_IN_BOUNDS(d, kSiteTokRow, row0, d.gk, quant_rows(d)) ||
      !KVQ_IN_BOUNDS(d, kSiteTokGroup, gidx, quant_groups(d)))
    row0 = gidx = 0;

  // ---- key (scale, zero): two channels and a slab of the tokens per thread, then over the slabs ----
  __half2* red = reinterpret_cast<__half2*>(vp);                 // [slab][channel pair][min, max]
  const int pairs = d.dk / 2, slabs = min(kThreads / pairs, d.gk);
  {
    const int p = tid % pairs, slab = tid / pairs;
    if (slab < slabs) {
      const __half* x = sk + slab * ks + 2 * p;
      __half2 mn = *reinterpret_cast<const __half2*>(x), mx = mn;
      for (int t = slab + slabs; t < d.gk; t += slabs) {
        const __half2 e = *reinterpret_cast<const __half2*>(sk + t * ks + 2 * p);
        mn = __hmin2(mn, e);
        mx = __hmax2(mx, e);
      }
      red[(slab * pairs + p) * 2] = mn;
      red[(slab * pairs + p) * 2 + 1] = mx;
    }
  }
  __syncthreads();
  for (int ch = tid; ch < d.dk; ch += kThreads) {
    int width = d.kb, off;
    if (d.var) channel_width(d.kcnt, ch, &width, &off);
    GroupParams gp;
    gp.scale = gp.zero = 0.0f;
    gp.sz = __floats2half2_rn(0.0f, 0.0f);
    if (width) {
      const __half* r = reinterpret_cast<const __half*>(red) + (ch / 2) * 4 + ch % 2;
      __half mn = r[0], mx = r[2];
      for (int sl = 1; sl < slabs; ++sl) {
        mn = __hmin(mn, r[sl * pairs * 4]);
        mx = __hmax(mx, r[sl * pairs * 4 + 2]);
      }
      gp = group_params_b(__half2float(mn), __half2float(mx), width);
    }
    kp[ch] = make_float2(gp.scale, gp.zero);
    kr[ch] = gp.scale == 0.0f ? 0.0f : __frcp_rn(gp.scale);
    __half* blk = reinterpret_cast<__half*>(c.ksz) + gidx * 2 * d.dk;
    const int at = d.var ? 2 * ch : key_slot(ch, d.dk, d.kb), to_zero = d.var ? 1 : 32 / d.kb;
    blk[at] = __low2half(gp.sz);
    blk[at + to_zero] = __high2half(gp.sz);
  }
  __syncthreads();

  // ---- values: 8 channels of a token per thread, a group's threads side by side in a warp ----
  {
    const int tpg = d.gv / 8;                                    // threads a group: a power of two, at most 32
    const int total = d.gk * vv;                                 // a multiple of 32: whole warps take part or none
    for (int i = tid; i < total; i += kThreads) {
      const int t = i / vv, cc = i % vv, vg = cc / tpg;
      const uint4 raw = *reinterpret_cast<const uint4*>(sv + t * vs + 8 * cc);
      const __half2* hx = reinterpret_cast<const __half2*>(&raw);
      __half2 mn = __hmin2(__hmin2(hx[0], hx[1]), __hmin2(hx[2], hx[3]));
      __half2 mx = __hmax2(__hmax2(hx[0], hx[1]), __hmax2(hx[2], hx[3]));
      for (int o = 1; o < tpg; o <<= 1) {
        mn = __hmin2(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = __hmax2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      }
      int width = d.vb, off = 8 * cc * d.vb;
      if (d.var) channel_width(d.vcnt, 8 * cc, &width, &off);
      GroupParams gp;
      gp.scale = gp.zero = 0.0f;
      gp.sz = __floats2half2_rn(0.0f, 0.0f);
      if (width)
        gp = group_params_b(__half2float(__hmin(__low2half(mn), __high2half(mn))),
                            __half2float(__hmax(__low2half(mx), __high2half(mx))), width);
      if (cc % tpg == 0) c.vsz[(row0 + t) * d.nvg + vg] = gp.sz;
      if (width == 0) continue;
      const uint64_t codes = chunk_codes(raw, width, [&](int) { return make_float3(gp.zero, gp.scale == 0.0f ? 0.0f : __frcp_rn(gp.scale), gp.scale); });
      store_codes(c.vcode + (row0 + t) * d.vw, off, 8 * width, codes);
    }
    if (d.var) zero_tail(d.vcnt, d.vw, c.vcode + row0 * d.vw, d.gk, tid);
  }

  // ---- key codes: 8 channels of a token per thread; of a width map, a word ----
  if (!d.var) {
    // d_k / 8 divides the CTA, so a thread keeps its chunk and the chunk's parameters
    const int cc = tid % vk;
    float3 prm[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) prm[j] = make_float3(kp[8 * cc + j].y, kr[8 * cc + j], kp[8 * cc + j].x);
    for (int t = tid / vk; t < d.gk; t += kThreads / vk) {
      const uint4 raw = *reinterpret_cast<const uint4*>(sk + t * ks + 8 * cc);
      const uint64_t codes = chunk_codes(raw, d.kb, [&](int j) { return prm[j]; });
      store_codes(c.kcode + (row0 + t) * d.kw, 8 * cc * d.kb, 8 * d.kb, codes);
    }
  } else {
    for (int i = tid; i < d.gk * d.kw; i += kThreads) {
      // the classes' channels (8, 4, 2, 1 bits) follow each other in the row; the word takes those
      // whose field starts inside it
      const int t = i / d.kw, wd = i % d.kw;
      uint32_t word = 0;
      int off = -32 * wd, ch = 0;
      for (int cl = 0; cl < 4 && off < 32; ++cl) {
        const int bits = 8 >> cl, skip = off < 0 ? min(d.kcnt[cl], -off / bits) : 0;
        off += skip * bits;
        const int end = ch + d.kcnt[cl];
        for (ch += skip; ch < end && off < 32; ++ch, off += bits) {
          GroupParams gp;
          gp.scale = kp[ch].x;
          gp.zero = kp[ch].y;
          word |= quant_code_b(__half2float(sk[t * ks + ch]), gp, bits) << off;
        }
      }
      c.kcode[(row0 + t) * d.kw + wd] = word;
    }
  }

  // ---- side code: the residual of every key projected on U_h, quantized per coordinate ----
  if (d.sr) {
    const float* u = c.side_u + static_cast<size_t>(h) * d.dk * d.sr;
    for (int i = tid; i < d.gk * d.sr; i += kThreads) {
      const int t = i / d.sr, r = i % d.sr;
      float acc = 0.0f;
      for (int ch = 0; ch < d.dk; ++ch) {
        GroupParams gp;
        gp.scale = kp[ch].x;
        gp.zero = kp[ch].y;
        const float x = __half2float(sk[t * ks + ch]);
        const float code = static_cast<float>(quant_code_b(x, gp, d.kb));
        const float e = __fsub_rn(x, __fadd_rn(__fmul_rn(code, gp.scale), gp.zero));
        acc = __fadd_rn(acc, __fmul_rn(e, u[ch * d.sr + r]));
      }
      y[t * d.sr + r] = acc;
    }
    __syncthreads();
    for (int r = tid; r < d.sr; r += kThreads) {
      float mn = y[r], mx = y[r];
      for (int t = 1; t < d.gk; ++t) {
        mn = fminf(mn, y[t * d.sr + r]);
        mx = fmaxf(mx, y[t * d.sr + r]);
      }
      const GroupParams gp = group_params_b(mn, mx, d.sq);
      zp[r] = make_float2(gp.scale, gp.zero);
      c.zsz[gidx * d.sr + r] = gp.sz;
    }
    __syncthreads();
    for (int t = tid; t < d.gk; t += kThreads) {
      uint32_t row = 0;
      for (int r = 0; r < d.sr; ++r) {
        GroupParams gp;
        gp.scale = zp[r].x;
        gp.zero = zp[r].y;
        row |= quant_code_b(y[t * d.sr + r], gp, d.sq) << (r * d.sq);
      }
      uint8_t* dst = c.zcode + (row0 + t) * d.zb;
      if (d.zb == 4)
        *reinterpret_cast<uint32_t*>(dst) = row;
      else
        *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(row);
    }
  }
}

// The new tokens that stay in the window, positions max(L, Q') .. L + n - 1: kRows rows a warp, the
// 16-byte pieces of their keys and values dealt to its lanes, all loads ahead of the stores.
constexpr int kRows = 4;
__global__ void __launch_bounds__(kThreads)
append_window_kernel(Dims d, CacheOut c, SeqChunk w, const __half* __restrict__ k, const __half* __restrict__ v,
                     int T, const int* __restrict__ index) {
  const int h = blockIdx.y, b = blockIdx.z, bh = b * d.Hkv + h;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqNew s = seq_new(w, b, d.log_retain);
  const int first = max(s.L, prefix_of(d, s.L + s.n)) + (blockIdx.x * (kThreads / 32) + warp) * kRows;
  const int rows = min(kRows, s.L + s.n - first);
  if (rows <= 0) return;
  const int vk = d.rot ? 0 : d.dk / 8, vv = d.dv / 8;      // (rotated keys go row by row below)
  for (int e = lane; e < vk + vv; e += 32) {
    uint4 x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i < rows) {
        const __half* src = e < vk ? token_source(d, nullptr, k, d.dk, index, T, s, b, bh, first + i).base + 8 * e
                                   : token_source(d, nullptr, v, d.dv, index, T, s, b, bh, first + i).base + 8 * (e - vk);
        x[i] = __ldg(reinterpret_cast<const uint4*>(src));
      }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long row = static_cast<long long>(bh) * d.cap + (first + i) % d.cap;
      if (i < rows && KVQ_IN_BOUNDS(d, kSiteTokWin, row, win_rows(d)))
        *reinterpret_cast<uint4*>(e < vk ? c.win_k + row * d.dk + 8 * e : c.win_v + row * d.dv + 8 * (e - vk)) = x[i];
    }
  }
  for (int i = 0; d.rot && i < rows; ++i) {
    const __half* pk = token_source(d, nullptr, k, d.dk, index, T, s, b, bh, first + i).base;
    const long long row = static_cast<long long>(bh) * d.cap + (first + i) % d.cap;
    if (!KVQ_IN_BOUNDS(d, kSiteTokWin, row, win_rows(d))) continue;
    float x[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) x[m] = m < d.dk / 32 ? __half2float(pk[lane + 32 * m]) : 0.0f;
    rotate_row_warp<8>(x, d.dk / 32, d.rot_signs, d.rot_inv_ck, lane);
#pragma unroll
    for (int m = 0; m < 8; ++m)
      if (m < d.dk / 32) c.win_k[row * d.dk + lane + 32 * m] = __float2half_rn(x[m]);
  }
}

}  // namespace

cudaError_t launch_append_tokens(const Dims& d, const CacheOut& c, const SeqChunk& w, const __half* k,
                                 const __half* v, int T, const int* index, int max_new_groups, int max_tail,
                                 cudaStream_t s) {
  if (max_new_groups > 0) {
    const size_t rows = static_cast<size_t>(d.gk) * (d.dk + d.dv + 2 * kPad) * 2;
    size_t smem = rows + d.dk * 12 + 4096 + d.gk * 32 + 64;
    smem = std::max(smem, static_cast<size_t>(kMaxRetained) * (d.dk + d.dv + 2 * kPad) * 2);
    static SmemLimit limit;
    const cudaError_t e = limit.raise(append_groups_kernel, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const dim3 grid(max_new_groups + (d.log_retain ? 1 : 0), d.Hkv, d.B);
    append_groups_kernel<<<grid, kThreads, smem, s>>>(d, c, w, k, v, T, index, max_new_groups);
    const cudaError_t e2 = cudaGetLastError();
    if (e2 != cudaSuccess) return e2;
  }
  if (max_tail > 0) {
    const int per_cta = kThreads / 32 * kRows;
    const dim3 grid((max_tail + per_cta - 1) / per_cta, d.Hkv, d.B);
    append_window_kernel<<<grid, kThreads, 0, s>>>(d, c, w, k, v, T, index);
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace kvq
