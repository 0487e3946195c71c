// Chunk attention on CUDA cores (any supported cache), and the parts that every chunk kernel
// shares: the merge of split partials and the rotation of query and new-key rows.
//
// A sequence's T new tokens (n valid) attend over its L cached tokens and over the new tokens
// that the mask lets them see:
//   o_t = sum_j 2^(s_tj - m) v_j / sum_j 2^(s_tj - m),   s_tj = log2(e) q_t.k_j / sqrt(d_k),
// the quantized keys and values being code * s + z, the side code adding (U_h^T q_t).z_j as in
// the one-token decode.  Row r = rep * T + t of a kv head's query block is query head
// h * n_rep + rep; a CTA takes kRows of those rows and one split of the tokens, a warp a token
// at a time: lanes hold d / 32 channels, dot products reduce by shuffles.  The tensor-core
// kernel takes over where it is built for the shape; this one serves everything else.
#include <algorithm>

#include "seq_ops.cuh"

namespace kvq {
namespace {

constexpr int kRows = 8;
constexpr int kMaxC = 8;      // d / 32, d <= 256
constexpr int kWarps = 4;

__global__ void __launch_bounds__(kWarps * 32)
chunk_simple_kernel(Dims d, CacheBufs cb, const __grid_constant__ ChunkArgs a) {
  __shared__ float sm_m[kWarps][kRows];
  __shared__ float sm_l[kWarps][kRows];
  __shared__ float sm_o[kWarps][kRows][kMaxC * 32];
  __shared__ float sm_qt[kRows][8];     // U_h^T q of each row, times the score scale

  const int split = blockIdx.x % a.splits, rb = blockIdx.x / a.splits, h = blockIdx.y, b = blockIdx.z;
  const int bh = b * d.Hkv + h;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ck = d.dk / 32, cv = d.dv / 32;
  const SeqNew sw = seq_new(a.seq, b, d.log_retain);
  if (sw.n == 0) return;
  const int n_rows = d.n_rep * a.T, r0 = rb * kRows, nr = min(kRows, n_rows - r0);

  float qr[kRows][kMaxC];
  const __half* qb = a.q + (static_cast<size_t>(bh) * n_rows + r0) * d.dk;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int j = 0; j < kMaxC; ++j)
      qr[r][j] = (r < nr && j < ck)
                     ? __half2float(qb[static_cast<size_t>(r) * d.dk + lane + 32 * j]) * a.score_scale : 0.0f;
  if (d.sr) {
    if (warp == 0) {
      const float* u = cb.side_u + static_cast<size_t>(h) * d.dk * d.sr;
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        for (int i = 0; i < d.sr; ++i) {
          float acc = 0.0f;
#pragma unroll
          for (int j = 0; j < kMaxC; ++j)
            if (j < ck) acc = fmaf(u[(lane + 32 * j) * d.sr + i], qr[r][j], acc);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
          if (lane == 0) sm_qt[r][i] = acc;
        }
    }
    __syncthreads();
  }
  float m[kRows], l[kRows], o[kRows][kMaxC];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxC; ++j) o[r][j] = 0.0f;
  }
  // widths and bit offsets of the lane's channels in a packed row: word << 16 | shift << 8 | width
  uint32_t kf[kMaxC], vf[kMaxC];
#pragma unroll
  for (int j = 0; j < kMaxC; ++j) {
    const int ch = lane + 32 * j;
    int wd = d.kb, off = ch * d.kb;
    if (d.var) channel_width(d.kcnt, ch, &wd, &off);
    kf[j] = j < ck && wd ? static_cast<uint32_t>(off / 32) << 16 | static_cast<uint32_t>(off % 32) << 8 | wd : 0u;
    wd = d.vb;
    off = ch * d.vb;
    if (d.var) channel_width(d.vcnt, ch, &wd, &off);
    vf[j] = j < cv && wd ? static_cast<uint32_t>(off / 32) << 16 | static_cast<uint32_t>(off % 32) << 8 | wd : 0u;
  }
  // tokens: the quantized prefix, the fp16 list (retained, window), the new ones
  const int n_old = sw.Q + sw.n_ret + (sw.L - sw.Q), n_all = n_old + sw.n;
  const int begin = a.new_only ? n_old : static_cast<int>(static_cast<long long>(split) * n_all / a.splits);
  const int end = static_cast<int>(static_cast<long long>(split + 1) * n_all / a.splits);
  const int mask_words = (a.T + 31) / 32;

  for (int i = begin + warp; i < end; i += kWarps) {
    float kh[kMaxC], vh[kMaxC], zhat[8];
    unsigned sees = (1u << nr) - 1u;        // rows of the block that see this token
#pragma unroll
    for (int j = 0; j < 8; ++j) zhat[j] = 0.0f;
    if (i < sw.Q) {
      if (d.log_retain && is_retained(sw.Q, i)) continue;      // read from the fp16 list
      const bool ok = KVQ_IN_BOUNDS(d, kSiteChunkTable, i / d.gk, d.max_groups);
      size_t row = ok ? group_row(d, cb.table, b, h, i / d.gk) + i % d.gk : 0;
      size_t gidx = ok ? group_index(d, cb.table, b, h, i / d.gk) : 0;
      if (!KVQ_IN_BOUNDS(d, kSiteChunkRow, static_cast<long long>(row), quant_rows(d)) ||
          !KVQ_IN_BOUNDS(d, kSiteChunkGroup, static_cast<long long>(gidx), quant_groups(d)))
        row = gidx = 0;
      if (d.sr) {
        const uint8_t* zr = cb.zcode + row * d.zb;
        const uint32_t zrow = d.zb == 4 ? *reinterpret_cast<const uint32_t*>(zr)
                                        : *reinterpret_cast<const uint16_t*>(zr);
        const __half2* zs = cb.zsz + gidx * d.sr;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < d.sr) {
            const float2 sz = __half22float2(zs[j]);
            zhat[j] = fmaf(static_cast<float>((zrow >> (j * d.sq)) & ((1u << d.sq) - 1u)), sz.x, sz.y);
          }
      }
      const uint32_t* kr = cb.kcode + row * d.kw;
      const uint32_t* vr = cb.vcode + row * d.vw;
      const __half* ks = reinterpret_cast<const __half*>(cb.ksz) + gidx * 2 * d.dk;
      const __half2* vs = cb.vsz + row * d.nvg;
#pragma unroll
      for (int j = 0; j < kMaxC; ++j) {
        const int ch = lane + 32 * j;
        kh[j] = vh[j] = 0.0f;
        if (kf[j]) {
          const uint32_t code = (kr[kf[j] >> 16] >> ((kf[j] >> 8) & 31u)) & ((1u << (kf[j] & 15u)) - 1u);
          int at = 2 * ch, to_zero = 1;
          if (!d.var) {     // the paired, quarter-interleaved block of a fixed-width group
            at = key_slot(ch, d.dk, d.kb);
            to_zero = 32 / d.kb;
          }
          kh[j] = fmaf(static_cast<float>(code), __half2float(ks[at]), __half2float(ks[at + to_zero]));
        }
        if (vf[j]) {
          const uint32_t code = (vr[vf[j] >> 16] >> ((vf[j] >> 8) & 31u)) & ((1u << (vf[j] & 15u)) - 1u);
          const float2 sz = __half22float2(vs[ch / d.gv]);
          vh[j] = fmaf(static_cast<float>(code), sz.x, sz.y);
        }
      }
    } else {
      const __half *kp, *vp;
      if (i < sw.Q + sw.n_ret) {
        size_t s = static_cast<size_t>(bh) * kMaxRetained + (i - sw.Q);
        if (!KVQ_IN_BOUNDS(d, kSiteChunkFp16, static_cast<long long>(s), ret_rows(d))) s = 0;
        kp = cb.ret_k + s * d.dk;
        vp = cb.ret_v + s * d.dv;
      } else if (i < n_old) {
        size_t s = static_cast<size_t>(bh) * d.cap + (i - sw.n_ret) % d.cap;     // position Q + (i - Q - n_ret)
        if (!KVQ_IN_BOUNDS(d, kSiteChunkFp16, static_cast<long long>(s), win_rows(d))) s = 0;
        kp = cb.win_k + s * d.dk;
        vp = cb.win_v + s * d.dv;
      } else {
        const int j = i - n_old;
        const size_t s = static_cast<size_t>(bh) * a.T + j;
        kp = a.k_new + s * d.dk;
        vp = a.v_new + s * d.dv;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int t = (r0 + r) % a.T;
          const bool see = a.mask ? t < sw.n && ((a.mask[(static_cast<size_t>(b) * a.T + t) * mask_words + j / 32] >>
                                                  (j % 32)) & 1u)
                                  : j <= t;
          if (!see) sees &= ~(1u << r);
        }
      }
#pragma unroll
      for (int j = 0; j < kMaxC; ++j) {
        kh[j] = j < ck ? __half2float(kp[lane + 32 * j]) : 0.0f;
        vh[j] = j < cv ? __half2float(vp[lane + 32 * j]) : 0.0f;
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (!((sees >> r) & 1u)) continue;                  // uniform per warp
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < kMaxC; ++j) s = fmaf(qr[r][j], kh[j], s);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (d.sr) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < d.sr) s = fmaf(sm_qt[r][j], zhat[j], s);
      }
      const float mn = fmaxf(m[r], s);
      const float alpha = exp2f(m[r] - mn);
      const float pe = exp2f(s - mn);
      l[r] = fmaf(l[r], alpha, pe);
#pragma unroll
      for (int j = 0; j < kMaxC; ++j) o[r][j] = fmaf(o[r][j], alpha, pe * vh[j]);
      m[r] = mn;
    }
  }

  // merge the CTA's warps; one split writes the output, several write partials
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (lane == 0) {
      sm_m[warp][r] = m[r];
      sm_l[warp][r] = l[r];
    }
#pragma unroll
    for (int j = 0; j < kMaxC; ++j)
      if (j < cv) sm_o[warp][r][lane + 32 * j] = o[r][j];
  }
  __syncthreads();
  for (int r = 0; r < nr; ++r) {
    if ((r0 + r) % a.T >= sw.n) continue;
    float M = -INFINITY;
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, sm_m[k][r]);
    const size_t row = static_cast<size_t>(bh) * n_rows + r0 + r;
    float wk[kWarps];
    float Lsum = 0.0f;
    for (int k = 0; k < kWarps; ++k) {
      wk[k] = (M == -INFINITY || sm_m[k][r] == -INFINITY) ? 0.0f : exp2f(sm_m[k][r] - M);
      Lsum = fmaf(wk[k], sm_l[k][r], Lsum);
    }
    const size_t part = row * a.splits + split;
    const bool partial = a.splits > 1 || a.new_only;
    if (partial && threadIdx.x == 0) a.ml[part] = make_float2(M, Lsum);
    for (int ch = threadIdx.x; ch < d.dv; ch += blockDim.x) {
      float acc = 0.0f;
      for (int k = 0; k < kWarps; ++k) acc = fmaf(wk[k], sm_o[k][r][ch], acc);
      if (partial)
        a.o[part * d.dv + ch] = acc;
      else
        a.out[row * d.dv + ch] = __float2half_rn(Lsum > 0.0f ? acc / Lsum : 0.0f);   // a row that sees nothing: 0
    }
  }
}

// Merge of a row's split partials, a warp per row: o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,
// 0 for a row that saw nothing; rows behind a sequence's new tokens are not written.
__global__ void __launch_bounds__(128)
chunk_combine_kernel(Dims d, const __grid_constant__ ChunkArgs a, long long rows) {
  // a programmatic dependent of the chunk kernel: its partials are visible behind this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int t = static_cast<int>(row % a.T);
  const int b = static_cast<int>(row / (static_cast<long long>(a.T) * d.Hq));
  if (t >= a.seq.n[a.seq.uniform ? 0 : b]) return;
  const float2* ml = a.ml + row * a.splits;
  const float* o = a.o + row * a.splits * d.dv;
  float M = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float den = 0.0f;
  float4 num[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  for (int s = 0; s < a.splits; ++s) {
    const float2 v = ml[s];
    const float w = v.x == -INFINITY ? 0.0f : exp2f(v.x - M);
    den = fmaf(w, v.y, den);
    if (w == 0.0f) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = 4 * lane + 128 * i;
      if (c < d.dv) {
        const float4 x = *reinterpret_cast<const float4*>(o + static_cast<size_t>(s) * d.dv + c);
        num[i].x = fmaf(w, x.x, num[i].x);
        num[i].y = fmaf(w, x.y, num[i].y);
        num[i].z = fmaf(w, x.z, num[i].z);
        num[i].w = fmaf(w, x.w, num[i].w);
      }
    }
  }
  const float inv = den > 0.0f ? 1.0f / den : 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = 4 * lane + 128 * i;
    if (c < d.dv) {
      const __half2 h0 = __floats2half2_rn(num[i].x * inv, num[i].y * inv);
      const __half2 h1 = __floats2half2_rn(num[i].z * inv, num[i].w * inv);
      uint2 packed;
      packed.x = *reinterpret_cast<const uint32_t*>(&h0);
      packed.y = *reinterpret_cast<const uint32_t*>(&h1);
      *reinterpret_cast<uint2*>(a.out + row * d.dv + c) = packed;
    }
  }
}

// q [B * Hq][T][dk] to [T][B * Hq][dk], 16 bytes a thread.
__global__ void __launch_bounds__(256)
step_queries_kernel(const uint4* __restrict__ q, uint4* __restrict__ steps, int rows, int T, int vec) {
  const long long n = static_cast<long long>(rows) * T * vec;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const int e = static_cast<int>(i % vec), t = static_cast<int>(i / vec % T);
    steps[(static_cast<long long>(t) * rows + i / vec / T) * vec + e] = q[i];
  }
}

// Merge of a row's decode-step partials (of tokens t0 to t0 + nt - 1) with that of its new tokens,
// a warp per row.
__global__ void __launch_bounds__(128)
combine_steps_kernel(Dims d, const __grid_constant__ ChunkArgs a, const float2* __restrict__ step_ml,
                     const float* __restrict__ step_o, int step_splits, int t0, int nt) {
  const int lane = threadIdx.x & 31;
  const int heads = d.B * d.Hq;
  const int i = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5);   // (token, sequence, head)
  if (i >= nt * heads) return;
  const int t = t0 + i / heads, bh = i % heads;
  if (t >= a.seq.n[a.seq.uniform ? 0 : bh / d.Hq]) return;
  const long long row = static_cast<long long>(bh) * a.T + t;
  const long long first = static_cast<long long>(i) * step_splits;
  float M = a.ml[row].x;
  for (int s = lane; s < step_splits; s += 32) M = fmaxf(M, step_ml[first + s].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float den = 0.0f, num[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s <= step_splits; ++s) {
    const float2 v = s < step_splits ? step_ml[first + s] : a.ml[row];
    const float* o = s < step_splits ? step_o + (first + s) * d.dv : a.o + row * d.dv;
    const float w = v.x == -INFINITY ? 0.0f : exp2f(v.x - M);
    den = fmaf(w, v.y, den);
    if (w == 0.0f) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < d.dv) num[i] = fmaf(w, o[lane + 32 * i], num[i]);
  }
  const float inv = den > 0.0f ? 1.0f / den : 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (lane + 32 * i < d.dv) a.out[row * d.dv + lane + 32 * i] = __float2half_rn(num[i] * inv);
}

__global__ void __launch_bounds__(256)
rotate_rows_kernel(Dims d, const __half* __restrict__ src, __half* __restrict__ dst, long long rows, float inv_c) {
  const int lane = threadIdx.x & 31;
  for (long long r = (blockIdx.x * 256LL + threadIdx.x) / 32; r < rows; r += gridDim.x * 8LL) {
    float x[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) x[m] = m < d.dk / 32 ? __half2float(src[r * d.dk + lane + 32 * m]) : 0.0f;
    rotate_row_warp<8>(x, d.dk / 32, d.rot_signs, inv_c, lane);
#pragma unroll
    for (int m = 0; m < 8; ++m)
      if (m < d.dk / 32) dst[r * d.dk + lane + 32 * m] = __float2half_rn(x[m]);
  }
}

}  // namespace

int chunk_simple_splits(const Dims& d, int L, int T, int num_splits) {
  const int most = std::min(64, std::max(1, (L + T) / 64));       // at least 64 tokens a split
  if (num_splits > 0) return std::min(num_splits, most);
  const long long ctas = static_cast<long long>(d.B) * d.Hkv * ((d.n_rep * T + kRows - 1) / kRows);
  const long long want = (8LL * d.sm_count + ctas - 1) / ctas;
  return static_cast<int>(std::min<long long>(want, most));
}

cudaError_t launch_chunk_simple(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  const int row_blocks = (d.n_rep * a.T + kRows - 1) / kRows;
  const dim3 grid(a.splits * row_blocks, d.Hkv, d.B);
  chunk_simple_kernel<<<grid, kWarps * 32, 0, s>>>(d, c, a);
  return cudaGetLastError();
}

cudaError_t launch_chunk_combine(const Dims& d, const ChunkArgs& a, cudaStream_t s) {
  const long long rows = static_cast<long long>(d.B) * d.Hq * a.T;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_combine_kernel, d, a, rows);
}

cudaError_t launch_step_queries(const Dims& d, const __half* q, __half* steps, int T, cudaStream_t s) {
  const long long n = static_cast<long long>(d.B) * d.Hq * T * (d.dk / 8);
  const unsigned ctas = static_cast<unsigned>(std::min<long long>((n + 255) / 256, 148 * 16));
  step_queries_kernel<<<ctas, 256, 0, s>>>(reinterpret_cast<const uint4*>(q), reinterpret_cast<uint4*>(steps),
                                           d.B * d.Hq, T, d.dk / 8);
  return cudaGetLastError();
}

cudaError_t launch_combine_steps(const Dims& d, const ChunkArgs& a, const float2* step_ml, const float* step_o,
                                 int step_splits, int t0, cudaStream_t s) {
  const int nt = std::min(kStepTokens, a.T - t0);
  const long long rows = static_cast<long long>(d.B) * d.Hq * nt;
  combine_steps_kernel<<<static_cast<unsigned>((rows + 3) / 4), 128, 0, s>>>(d, a, step_ml, step_o, step_splits, t0, nt);
  return cudaGetLastError();
}

cudaError_t launch_rotate_rows(const Dims& d, const __half* src, __half* dst, long long rows, float inv_c,
                               cudaStream_t s) {
  const long long ctas = (rows + 7) / 8;
  rotate_rows_kernel<<<static_cast<unsigned>(ctas < 148 * 16 ? ctas : 148 * 16), 256, 0, s>>>(d, src, dst, rows, inv_c);
  return cudaGetLastError();
}

}  // namespace kvq
