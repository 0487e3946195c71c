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
    t.base = fresh + (static_cast<long long>(bh) * T + r) * width;
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

// Half index of (scale, zero) of channel c in a fixed-width key group's block.
__device__ __forceinline__ int key_slot(int c, int dk, int kb) {
  const int per = 32 / kb, half = per / 2, words = dk / per, quarter = words % 4 == 0 ? words / 4 : 0;
  const int w = c / per, r = c % per, pos = quarter ? (w % quarter) * 4 + w / quarter : w;
  return pos * 2 * per + (r % half) * 2 + r / half;
}

__global__ void __launch_bounds__(kThreads)
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
  // shared memory: key rows, value rows, key (scale, zero), value (scale, zero), side residual sums,
  // side (scale, zero)
  __half* sk = reinterpret_cast<__half*>(smem);
  __half* sv = sk + d.gk * ks;
  float2* kp = reinterpret_cast<float2*>(sv + d.gk * vs);
  float2* vp = kp + d.dk;
  float* y = reinterpret_cast<float*>(vp + d.gk * d.nvg);
  float2* zp = reinterpret_cast<float2*>(y + d.gk * 8);
  const int p0 = g * d.gk;
  for (int t = warp; t < d.gk; t += nwarps) {
    const TokenSource a = token_source(d, c.win_k, k, d.dk, index, T, s, b, bh, p0 + t);
    const TokenSource e2 = token_source(d, c.win_v, v, d.dv, index, T, s, b, bh, p0 + t);
    for (int e = lane; e < vk; e += 32)
      reinterpret_cast<uint4*>(sk + t * ks)[e] = reinterpret_cast<const uint4*>(a.base)[e];
    for (int e = lane; e < vv; e += 32)
      reinterpret_cast<uint4*>(sv + t * vs)[e] = reinterpret_cast<const uint4*>(e2.base)[e];
    __syncwarp();
    if (a.fresh && d.rot) rotate_smem_row(sk + t * ks, d, lane);
  }
  __syncthreads();
  long long row0 = static_cast<long long>(group_row(d, c.table, b, h, g));
  long long gidx = static_cast<long long>(group_index(d, c.table, b, h, g));
  if (!KVQ_RANGE_IN_BOUNDS(d, kSiteTokRow, row0, d.gk, quant_rows(d)) ||
      !KVQ_IN_BOUNDS(d, kSiteTokGroup, gidx, quant_groups(d)))
    row0 = gidx = 0;

  // ---- (scale, zero): keys per channel, values per token and channel group ----
  for (int i = tid; i < d.dk + d.gk * d.nvg; i += kThreads) {
    const bool key = i < d.dk;
    const int t = key ? 0 : (i - d.dk) / d.nvg, vg = key ? 0 : (i - d.dk) % d.nvg;
    int width = key ? d.kb : d.vb, off;
    if (d.var) channel_width(key ? d.kcnt : d.vcnt, key ? i : vg * d.gv, &width, &off);
    GroupParams gp;
    gp.scale = gp.zero = 0.0f;
    gp.sz = __floats2half2_rn(0.0f, 0.0f);
    if (width) {
      const __half* x = key ? sk + i : sv + t * vs + vg * d.gv;
      const int n = key ? d.gk : d.gv, step = key ? ks : 1;
      __half mn = x[0], mx = x[0];
      for (int j = 1; j < n; ++j) {
        const __half e = x[j * step];
        mn = __hmin(mn, e);
        mx = __hmax(mx, e);
      }
      gp = group_params_b(__half2float(mn), __half2float(mx), width);
    }
    if (key) {
      kp[i] = make_float2(gp.scale, gp.zero);
      __half* blk = reinterpret_cast<__half*>(c.ksz) + gidx * 2 * d.dk;
      const int at = d.var ? 2 * i : key_slot(i, d.dk, d.kb), to_zero = d.var ? 1 : 32 / d.kb;
      blk[at] = __low2half(gp.sz);
      blk[at + to_zero] = __high2half(gp.sz);
    } else {
      vp[i - d.dk] = make_float2(gp.scale, gp.zero);
      c.vsz[(row0 + t) * d.nvg + vg] = gp.sz;
    }
  }
  __syncthreads();

  // ---- codes ----
  for (int i = tid; i < d.gk * (d.kw + d.vw); i += kThreads) {
    const bool key = i < d.gk * d.kw;
    const int j = key ? i : i - d.gk * d.kw;
    const int words = key ? d.kw : d.vw, t = j / words, wd = j % words;
    auto code = [&](int ch, int bits) {
      const float2 sz = key ? kp[ch] : vp[t * d.nvg + ch / d.gv];
      GroupParams gp;
      gp.scale = sz.x;
      gp.zero = sz.y;
      return quant_code_b(__half2float(key ? sk[t * ks + ch] : sv[t * vs + ch]), gp, bits);
    };
    uint32_t word = 0;
    if (d.var) {
      // a width map: the classes' channels (8, 4, 2, 1 bits) follow each other in the row; the
      // word takes those whose field starts inside it
      const int* cnt = key ? d.kcnt : d.vcnt;
      int off = -32 * wd, ch = 0;
      for (int cl = 0; cl < 4 && off < 32; ++cl) {
        const int bits = 8 >> cl, skip = off < 0 ? min(cnt[cl], -off / bits) : 0;
        off += skip * bits;
        const int end = ch + cnt[cl];
        for (ch += skip; ch < end && off < 32; ++ch, off += bits) word |= code(ch, bits) << off;
      }
    } else {
      const int bits = key ? d.kb : d.vb, per = 32 / bits;
      for (int e = 0; e < per; ++e) word |= code(wd * per + e, bits) << (e * bits);
    }
    (key ? c.kcode : c.vcode)[(row0 + t) * words + wd] = word;
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

// The new tokens that stay in the window, a warp per row: positions max(L, Q') .. L + n - 1.
__global__ void __launch_bounds__(kThreads)
append_window_kernel(Dims d, CacheOut c, SeqChunk w, const __half* __restrict__ k, const __half* __restrict__ v,
                     int T, const int* __restrict__ index) {
  const int h = blockIdx.y, b = blockIdx.z, bh = b * d.Hkv + h;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqNew s = seq_new(w, b, d.log_retain);
  const int Q2 = prefix_of(d, s.L + s.n);
  const int p = max(s.L, Q2) + blockIdx.x * (kThreads / 32) + warp;
  if (p >= s.L + s.n) return;
  const __half* pk = token_source(d, nullptr, k, d.dk, index, T, s, b, bh, p).base;
  const __half* pv = token_source(d, nullptr, v, d.dv, index, T, s, b, bh, p).base;
  const long long row = static_cast<long long>(bh) * d.cap + p % d.cap;
  if (!KVQ_IN_BOUNDS(d, kSiteTokWin, row, win_rows(d))) return;
  if (d.rot) {
    float x[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) x[m] = m < d.dk / 32 ? __half2float(pk[lane + 32 * m]) : 0.0f;
    rotate_row_warp<8>(x, d.dk / 32, d.rot_signs, d.rot_inv_ck, lane);
#pragma unroll
    for (int m = 0; m < 8; ++m)
      if (m < d.dk / 32) c.win_k[row * d.dk + lane + 32 * m] = __float2half_rn(x[m]);
  } else {
    for (int e = lane; e < d.dk / 8; e += 32)
      reinterpret_cast<uint4*>(c.win_k + row * d.dk)[e] = reinterpret_cast<const uint4*>(pk)[e];
  }
  for (int e = lane; e < d.dv / 8; e += 32)
    reinterpret_cast<uint4*>(c.win_v + row * d.dv)[e] = reinterpret_cast<const uint4*>(pv)[e];
}

}  // namespace

cudaError_t launch_append_tokens(const Dims& d, const CacheOut& c, const SeqChunk& w, const __half* k,
                                 const __half* v, int T, const int* index, int max_new_groups, int max_tail,
                                 cudaStream_t s) {
  if (max_new_groups > 0) {
    const size_t rows = static_cast<size_t>(d.gk) * (d.dk + d.dv + 2 * kPad) * 2;
    size_t smem = rows + d.dk * 8 + static_cast<size_t>(d.gk) * d.nvg * 8 + d.gk * 32 + 64;
      smem = std::max(smem, static_cast<size_t>(kMaxRetained) * (d.dk + d.dv + 2 * kPad) * 2);
    const cudaError_t e = cudaFuncSetAttribute(append_groups_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const dim3 grid(max_new_groups + (d.log_retain ? 1 : 0), d.Hkv, d.B);
    append_groups_kernel<<<grid, kThreads, smem, s>>>(d, c, w, k, v, T, index, max_new_groups);
    const cudaError_t e2 = cudaGetLastError();
    if (e2 != cudaSuccess) return e2;
  }
  if (max_tail > 0) {
    const dim3 grid((max_tail + kThreads / 32 - 1) / (kThreads / 32), d.Hkv, d.B);
    append_window_kernel<<<grid, kThreads, 0, s>>>(d, c, w, k, v, T, index);
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace kvq
