// Internal declarations of the operators on several tokens per sequence and on whole
// sequences: chunk attention, multi-token append, forks and page moves.
#pragma once

#include "kvq_internal.cuh"
#include "smem_limit.h"

namespace kvq {

// Lengths and new tokens of the sequences of one call (a launch parameter): sequence b holds
// L[b] tokens, Q[b] of them quantized, and brings n[b] new ones (one entry for all sequences
// when `uniform`).
struct SeqChunk {
  int uniform;
  int L[kMaxSeqs], Q[kMaxSeqs], n[kMaxSeqs];
};
struct SeqNew {
  int L, Q, n, n_ret;
};
__device__ __forceinline__ SeqNew seq_new(const SeqChunk& w, int b, int log_retain) {
  const int i = w.uniform ? 0 : b;
  SeqNew s;
  s.L = w.L[i];
  s.Q = w.Q[i];
  s.n = w.n[i];
  s.n_ret = log_retain ? retained_count(s.Q) : 0;
  return s;
}

// Quantized prefix of a sequence of L tokens.
__host__ __device__ inline int prefix_of(const Dims& d, int L) {
  if (d.kb == 16) return 0;
  const int over = L - d.R;
  return over > 0 ? over / d.gk * d.gk : 0;
}

// Position of word w of a key row of `words` words in its group's (scale, zero) block: the words'
// parts stand in the order of the row, or quarter-interleaved where 4 divides them.
__host__ __device__ constexpr int key_block_pos(int words, int w) {
  return words % 4 == 0 ? w % (words / 4) * 4 + w / (words / 4) : w;
}
// Half index of the scale of channel c in a fixed-width key group's block; its zero is 32 / kb
// further on.
__host__ __device__ constexpr int key_slot(int c, int dk, int kb) {
  const int per = 32 / kb, half = per / 2, r = c % per;
  return key_block_pos(dk / per, c / per) * 2 * per + (r % half) * 2 + r / half;
}

// Whether position p < Q is one of the retained tokens of a quantized prefix of Q tokens.
__device__ __forceinline__ bool is_retained(int Q, int p) {
  return (p & ((1 << (31 - __clz(Q - p))) - 1)) == 0;
}

// Device views of the cache buffers for the operators that write them.
struct CacheOut {
  uint32_t* kcode;
  __half2* ksz;
  uint32_t* vcode;
  __half2* vsz;
  __half* win_k;
  __half* win_v;
  __half* ret_k;
  __half* ret_v;
  uint8_t* zcode;
  __half2* zsz;
  const float* side_u;
  int* table;
};

// ---- multi-token append (append_tokens.cu) ----
// index: device int32 [B][T], the row of k / v that token i of a sequence is (null: row i).
// max_groups_out / max_tail: the most groups any sequence quantizes, the most rows it keeps.
cudaError_t launch_append_tokens(const Dims& d, const CacheOut& c, const SeqChunk& w, const __half* k,
                                 const __half* v, int T, const int* index, int max_new_groups, int max_tail,
                                 cudaStream_t s);

// ---- forks and page moves (pages.cu) ----
struct ForkList {
  int n;
  int src[kMaxSeqs], dst[kMaxSeqs], L[kMaxSeqs], Q[kMaxSeqs];
};
cudaError_t launch_fork(const Dims& d, const CacheOut& c, const ForkList& f, cudaStream_t s);

// One batch of a compaction: pages to copy, and block-table entries to write.  Launch parameters:
// a short batch (most pools) is a tenth of the copying that a launch does with a full one.
template <int CAP>
struct PageMovesT {
  int n_moves, n_writes;
  int src[CAP], dst[CAP];
  int idx[CAP], page[CAP];
};
constexpr int kFewMoves = 192, kMostMoves = 1984;     // four lists within 32 KB of parameters
using PageMoves = PageMovesT<kMostMoves>;
cudaError_t launch_page_moves(const Dims& d, const CacheOut& c, const PageMoves& m, cudaStream_t s);

// ---- chunk attention ----
// T query rows per head; a kv head's block of queries is n_rep * T contiguous rows, row
// r = rep * T + t.  Splits of a (b, kv head, row block) write (m, l) and unnormalised outputs
// per row to the workspace; one split writes `out` itself.
struct ChunkArgs {
  SeqChunk seq;
  int T;                  // query rows per head, and rows per head of k_new / v_new
  int splits, splits_q;   // all of them; of those over the quantized groups (few-row kernel)
  float score_scale;      // log2(e) / sqrt(d_k)
  const __half* q;        // [B][Hq][T][dk], rotated when the keys are
  const __half* k_new;    // [B][Hkv][T][dk], likewise
  const __half* v_new;    // [B][Hkv][T][dv]
  const uint32_t* mask;   // [B][T][ceil(T / 32)], bit j of row t: t sees new token j; null: causal
  __half* out;            // [B][Hq][T][dv]
  float2* ml;             // [B * Hq * T][splits]
  float* o;               // [B * Hq * T][splits][dv]
  unsigned int* status;
  int new_only;           // the CUDA-core kernel: the new tokens alone, as the partial of a row (splits 1)
};

// A width map's chunk runs as decode steps (one per new token) over the cached tokens, partials
// [kStepTokens][B * Hq][splits] of kStepTokens tokens at a time (the workspace does not grow with
// the prompt), and the CUDA-core kernel over the new ones, partials ml, o of ChunkArgs.
constexpr int kStepTokens = 16;
cudaError_t launch_step_queries(const Dims& d, const __half* q, __half* steps, int T, cudaStream_t s);
cudaError_t launch_combine_steps(const Dims& d, const ChunkArgs& a, const float2* step_ml, const float* step_o,
                                 int step_splits, int t0, cudaStream_t s);

// Splits of each (b, kv head, row block) for sequences of at most L cached tokens (num_splits > 0: that
// many, clamped to the tokens), for either kernel.
int chunk_simple_splits(const Dims& d, int L, int T, int num_splits);
int chunk_mma_splits(const Dims& d, int L, int T, int num_splits);
bool chunk_mma_supported(const Dims& d);
// One or a few new tokens, up to 24 query rows of a kv head, or a cache with a side code (chunk_few.cuh).
bool chunk_few_supported(const Dims& d, int T);
// Query rows that a block of the few-row kernel takes, of `rows` in all: half an n-tile of 8 columns (two
// columns a row), or one to three of them.
// With a side code three tiles spill about 580 bytes a thread (4-bit keys), but two blocks of 16 read
// the cache twice: 24 rows over 16 x 16k 198 us and 265, 4 x 32k 105 and 155, 16 x 1k 48 and 70 (8 kv
// heads; in between, from 4 sequences on, either is ahead, 16 x 2k 80 and 80, 4 x 4k 48 and 41).  Up to
// 3 sequences two blocks are: 1 x 4k 36 and 30, 1 x 32k 60 and 56, 3 x 8k 52 and 44.  Without a side
// code the other side of the rule is the narrow kernel.
inline int chunk_few_block(const Dims& d, int rows) {
  if (rows <= 8) return rows <= 4 ? 4 : 8;
  if (rows <= 16 || rows > 24) return 16;
  return d.sr && 6 * d.B * d.Hkv <= d.sm_count ? 16 : 24;
}
cudaError_t launch_chunk_few(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s);
// Up to this many query rows of a kv head the tokens take the MMA's rows (chunk_narrow.cu); with 64
// rows the narrow kernel's softmax took 1.40 ms where the wide one takes 0.85 (32 sequences of 32k).
constexpr int kNarrowRows = 32;
cudaError_t launch_chunk_narrow(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s);
cudaError_t launch_chunk_mma(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s);
cudaError_t launch_chunk_simple(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s);
cudaError_t launch_chunk_combine(const Dims& d, const ChunkArgs& a, cudaStream_t s);
// dst rows = rotations of src rows (rows of dk), scaled by inv_c
cudaError_t launch_rotate_rows(const Dims& d, const __half* src, __half* dst, long long rows, float inv_c,
                               cudaStream_t s);

}  // namespace kvq
