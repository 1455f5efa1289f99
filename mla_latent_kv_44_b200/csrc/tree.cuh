// Declarations shared by the kernels of mla_decode_tree.
#pragma once

#include "common.cuh"

namespace mla {

constexpr int kTreeTile = 128;      // query rows of a tile on the tensor-core path
constexpr int kTreeMaxSplits = 64;  // ranges of a sequence's cache rows on the CUDA-core path

// Everything the stages of mla_decode_tree need, resolved to device pointers.
struct TreeParams {
  const void* q;
  const void* pool;
  const int32_t* table;
  const int32_t* seq_lens;
  const uint32_t* mask;  // null: a chain
  float* lse;            // may be null
  uint32_t* err;
  float* part_o;    // partial results of split key ranges
  float* part_lse;
  int32_t H, r, dr, D, bs, max_blocks, num_blocks, batch, T, BT, words;
  float scale;
  // CUDA-core path: query rows per tile, tiles per sequence, key ranges per sequence
  int32_t tile_rows, tiles, splits;
  // tensor-core path: items are a sequence's groups of `team` tiles
  int32_t team, groups, ranges;
  // finished latent sums (BT, H, r) as two bf16 terms, hi = bf16(x) and lo = bf16(x - hi): 16 bits
  // of x in the operand type of the product with W_UV
  __nv_bfloat16 *latent_hi, *latent_lo;
  int4* cuts;  // per range: an item that goes on from the range before into this one (x; -1:
               // none that begins there), its pieces (y) and the slot of the first (z); piece
               // k > 0 is in slot 2 * (z / 2 + k)
};

// Longest sequence: row numbers rounded up to whole tiles stay below 2^31.
constexpr int kTreeMaxLen = 0x7fffffff - 8192;

// Rows of sequence b, its drafted ones included: 0 for an empty place of the batch and for a
// length that cannot be (fewer rows than drafted tokens, or more than the table holds), which
// `report` flags.
__device__ __forceinline__ int tree_length(const TreeParams& p, int b, bool report) {
  const int len = p.seq_lens[b];
  if (len >= p.T && len <= kTreeMaxLen && (int64_t)len <= (int64_t)p.max_blocks * p.bs) return len;
  if (len != 0 && report) set_error(p.err, MLA_DEV_BAD_LENGTH);
  return 0;
}

// Whether token t of sequence b attends drafted node `node` (0 <= node < T).
__device__ __forceinline__ bool tree_sees(const TreeParams& p, int b, int t, int node) {
  if (!p.mask) return node <= t;
  return (p.mask[((size_t)b * p.T + t) * p.words + (node >> 5)] >> (node & 31)) & 1u;
}

// First chunk of range q of R over C chunks, floor(q C / R); a 32-bit division, which takes a
// fraction of the time, where that is enough.
__host__ __device__ __forceinline__ int first_chunk(int q, int R, int C) {
  if (C < 1 << 25) return (int)((uint32_t)q * (uint32_t)C / (uint32_t)R);
  return (int)((int64_t)q * C / R);
}
static_assert(kRanges <= 127, "q C below 2^32");

cudaError_t launch_tree_simt(const mla_config& c, const TreeParams& p, const void* w_uv, void* o,
                             cudaStream_t st);
int tree_simt_tile_rows(const mla_config& c);
bool tree_tc_supported(const mla_config& c);
void tree_team(int tiles, int* team, int* ranges);
cudaError_t launch_tree_tc(const TreeParams& p, cudaStream_t st);
// tree_out.cu
cudaError_t launch_tree_out(const TreeParams& p, const void* w_uv, int dv, void* o,
                            cudaStream_t st);

// step_tables.cu
cudaError_t launch_build_tables(const int32_t* seq_lens, const int32_t* new_lens, int batch,
                                int32_t* table, int max_blocks, int bs, const int32_t* held,
                                int32_t* free_blocks, const int32_t* free_count, int num_blocks,
                                int32_t* held_out, int32_t* free_count_out, int32_t* cu,
                                int32_t* seq_idx, int32_t* pos, int64_t* slots, int max_tokens,
                                uint32_t* err, cudaStream_t st);
cudaError_t launch_tree_masks(const int32_t* parents, int parents_batch, const int32_t* seq_lens,
                              int batch, int T, uint32_t* mask, int32_t* pos, uint32_t* err,
                              cudaStream_t st);
// tree_cache.cu
cudaError_t launch_append_slots(const mla_config& c, const void* ckv, const void* kr,
                                const float* gamma, const int32_t* pos, const int64_t* slots,
                                void* pool, int num_blocks, int n, uint32_t* err,
                                cudaStream_t st);
cudaError_t launch_commit_tree(const mla_config& c, const int32_t* path, const int32_t* count,
                               int width, int T, const int32_t* table, int max_blocks, void* pool,
                               int num_blocks, const int32_t* seq_lens, int32_t* seq_lens_out,
                               int batch, uint32_t* err, cudaStream_t st);

}  // namespace mla
