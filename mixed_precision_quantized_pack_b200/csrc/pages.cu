// Forks of sequences and moves of pages: plain copies, bound by the bytes they move.
//
// A quantized group never changes once it is written, so a paged fork shares the parent's
// pages and copies only its block-table entries; the fp16 window and retained rows, which every
// sequence goes on writing, are copied.  Every span (a group array of one head, a run of
// window slots, an array of one page) starts on 16 bytes and is a multiple of 16 bytes long:
// CTAs walk it with four independent 16-byte loads per thread in flight.
#include <algorithm>

#include "seq_ops.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// bytes (a multiple of 16) from src to dst by the CTAs part, part + parts, ... of a span.
__device__ __forceinline__ void copy_span(const void* src, void* dst, size_t bytes, int part, int parts) {
  const uint4* s = static_cast<const uint4*>(src);
  uint4* t = static_cast<uint4*>(dst);
  const size_t n = bytes / 16, tile = kThreads * kUnroll;
  for (size_t i0 = part * tile; i0 < n; i0 += parts * tile) {
    uint4 x[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const size_t i = i0 + j * kThreads + threadIdx.x;
      if (i < n) x[j] = s[i];
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const size_t i = i0 + j * kThreads + threadIdx.x;
      if (i < n) t[i] = x[j];
    }
  }
}

// grid (parts, Hkv, pairs): pair z of the list, kv head y.
__global__ void __launch_bounds__(kThreads) fork_kernel(Dims d, CacheOut c, ForkList f) {
  const int h = blockIdx.y, i = blockIdx.z, part = blockIdx.x, parts = gridDim.x;
  const int src = f.src[i], dst = f.dst[i], L = f.L[i], Q = f.Q[i];
  if (!KVQ_IN_BOUNDS(d, kSiteForkSrc, src, d.B) || !KVQ_IN_BOUNDS(d, kSiteForkDst, dst, d.B)) return;
  const size_t sb = static_cast<size_t>(src) * d.Hkv + h, db = static_cast<size_t>(dst) * d.Hkv + h;
  // [row0, row0 + rows) of region sb to the same rows of region db; `row_bytes` per row, `cap` rows a region
  auto rows = [&](auto* base, size_t cap, size_t row_bytes, size_t row0, size_t n) {
    if (!base || n == 0) return;
    char* p = reinterpret_cast<char*>(base);
    copy_span(p + (sb * cap + row0) * row_bytes, p + (db * cap + row0) * row_bytes, n * row_bytes, part, parts);
  };
  if (d.paged) {
    if (h == 0 && part == 0)
      for (int g = threadIdx.x; g < Q / d.gk; g += kThreads)
        c.table[static_cast<size_t>(dst) * d.max_groups + g] = c.table[static_cast<size_t>(src) * d.max_groups + g];
  } else if (Q) {
    rows(c.kcode, d.lcap, d.kw * 4, 0, Q);
    rows(c.ksz, d.max_groups, d.dk * 4, 0, Q / d.gk);
    rows(c.vcode, d.lcap, d.vw * 4, 0, Q);
    rows(c.vsz, d.lcap, d.nvg * 4, 0, Q);
    if (d.sr) {
      rows(c.zcode, d.lcap, d.zb, 0, Q);
      rows(c.zsz, d.max_groups, d.sr * 4, 0, Q / d.gk);
    }
  }
  // the live slots of the window's ring: positions Q .. L - 1, in at most two runs
  const int first = Q % d.cap, head = min(L - Q, d.cap - first), tail = L - Q - head;
  rows(c.win_k, d.cap, d.dk * 2, first, head);
  rows(c.win_v, d.cap, d.dv * 2, first, head);
  rows(c.win_k, d.cap, d.dk * 2, 0, tail);
  rows(c.win_v, d.cap, d.dv * 2, 0, tail);
  if (d.log_retain) {
    rows(c.ret_k, kMaxRetained, d.dk * 2, 0, retained_count(Q));
    rows(c.ret_v, kMaxRetained, d.dv * 2, 0, retained_count(Q));
  }
}

// grid (moves + CTAs for the table entries, parts): CTA x < n_moves copies page src[x].
template <int CAP>
__global__ void __launch_bounds__(kThreads)
page_moves_kernel(Dims d, CacheOut c, const __grid_constant__ PageMovesT<CAP> m) {
  const int x = blockIdx.x;
  if (x >= m.n_moves) {
    const int i = (x - m.n_moves) * kThreads + threadIdx.x;
    if (blockIdx.y == 0 && i < m.n_writes &&
        KVQ_IN_BOUNDS(d, kSiteTableIdx, m.idx[i], static_cast<long long>(d.B) * d.max_groups) &&
        KVQ_IN_BOUNDS(d, kSiteTablePage, m.page[i], d.n_pages))
      c.table[m.idx[i]] = m.page[i];
    return;
  }
  const int src = m.src[x], dst = m.dst[x];
  if (!KVQ_IN_BOUNDS(d, kSitePageSrc, src, d.n_pages) || !KVQ_IN_BOUNDS(d, kSitePageDst, dst, d.n_pages)) return;
  auto page = [&](auto* base, size_t bytes) {
    if (!base) return;
    char* p = reinterpret_cast<char*>(base);
    copy_span(p + src * bytes, p + dst * bytes, bytes, blockIdx.y, gridDim.y);
  };
  const size_t rows = static_cast<size_t>(d.Hkv) * d.gk;
  page(c.kcode, rows * d.kw * 4);
  page(c.vcode, rows * d.vw * 4);
  page(c.ksz, static_cast<size_t>(d.Hkv) * d.dk * 4);
  page(c.vsz, rows * d.nvg * 4);
  if (d.sr) {
    page(c.zcode, rows * d.zb);
    page(c.zsz, static_cast<size_t>(d.Hkv) * d.sr * 4);
  }
}

}  // namespace

cudaError_t launch_fork(const Dims& d, const CacheOut& c, const ForkList& f, cudaStream_t s) {
  if (f.n < 1) return cudaSuccess;
  // enough CTAs per (pair, head) that the longest span keeps every SM busy, no more than it has tiles
  int longest = 0;
  for (int i = 0; i < f.n; ++i) longest = std::max(longest, d.paged ? f.L[i] - f.Q[i] : f.L[i]);
  const long long tiles = (static_cast<long long>(longest) * (d.kb == 16 || d.paged ? d.dk * 2 : d.kw * 4) +
                           16 * kThreads * kUnroll - 1) / (16 * kThreads * kUnroll);
  const long long want = (8LL * d.sm_count + static_cast<long long>(d.Hkv) * f.n - 1) / (static_cast<long long>(d.Hkv) * f.n);
  const dim3 grid(static_cast<unsigned>(std::max(1LL, std::min(tiles, want))), d.Hkv, f.n);
  fork_kernel<<<grid, kThreads, 0, s>>>(d, c, f);
  return cudaGetLastError();
}

cudaError_t launch_page_moves(const Dims& d, const CacheOut& c, const PageMoves& m, cudaStream_t s) {
  const int table_ctas = (m.n_writes + kThreads - 1) / kThreads;
  if (m.n_moves + table_ctas == 0) return cudaSuccess;
  const int want = m.n_moves ? (8 * d.sm_count + m.n_moves - 1) / m.n_moves : 1;
  const dim3 grid(m.n_moves + table_ctas, std::max(1, std::min(want, 8)));
  if (m.n_moves <= kFewMoves && m.n_writes <= kFewMoves) {
    PageMovesT<kFewMoves> f;
    f.n_moves = m.n_moves;
    f.n_writes = m.n_writes;
    std::copy_n(m.src, m.n_moves, f.src);
    std::copy_n(m.dst, m.n_moves, f.dst);
    std::copy_n(m.idx, m.n_writes, f.idx);
    std::copy_n(m.page, m.n_writes, f.page);
    page_moves_kernel<kFewMoves><<<grid, kThreads, 0, s>>>(d, c, f);
  } else {
    page_moves_kernel<kMostMoves><<<grid, kThreads, 0, s>>>(d, c, m);
  }
  return cudaGetLastError();
}

}  // namespace kvq
