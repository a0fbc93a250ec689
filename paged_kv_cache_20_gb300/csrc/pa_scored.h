// pa_scored.h -- launch entry points of scored attention (host code only).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct DecodeArgs;
struct CombineArgs;

// The second part of scored attention: weights from the scores and the rows'
// statistics, added to the ledger.
struct LedgerArgs {
  float *scores;              // [num_seqs][num_kv_heads][max_rows]
  int32_t *row_pos;           // the same shape, or nullptr
  const int32_t *seq_lens;    // [num_seqs] (with row_pos)
  const int32_t *context_lens, *block_tables;
  const float *raw_scores;    // [num_seqs][num_kv_heads][max_tiles][rows][16]
  const float *ws_m, *ws_l;   // [num_seqs][splits][q_len * num_q_heads]
  // the scores again from K and q (more than 16 query tokens), with the rows'
  // -(m + log2 l) [num_seqs][num_kv_heads][rows]
  const float *row_nlse;
  const void *q, *k_cache;
  const float *k_scale;
  float scale_log2;
  int num_seqs, num_kv_heads, group, q_len, rows, splits;  // rows = group * q_len
  int max_rows, max_tiles, block_size, max_blocks_per_seq, num_blocks;
  unsigned *err;
};

// After a decode pass that left its scores: the ledger, and with `combine` the merge of
// the partitions into the output, in one launch.
cudaError_t launch_finish(const LedgerArgs &args, const CombineArgs *combine, int head_dim, bool fp16,
                          cudaStream_t stream);
// Many query rows: the scores again from K and q on the tensor cores.  qmap: tensor map
// over q with a box of 64 columns x the heads x the tokens that mass_q_box names.  At
// most mass_max_seqs() sequences per launch.
cudaError_t launch_mass(const CUtensorMap &qmap, const LedgerArgs &args, int head_dim, bool fp16,
                        bool kv8, cudaStream_t stream);
void mass_q_box(int group, int *heads, int *tokens);
int mass_max_seqs();

// The decode kernels with their scores written to args.raw_scores; the single pass
// also writes its statistics.
cudaError_t launch_decode_scored_fp16(const CUtensorMap &kmap, const CUtensorMap &vmap,
                                      const DecodeArgs &args, int head_dim, bool kv8, bool partial,
                                      int units, cudaStream_t stream);
cudaError_t launch_decode_scored_bf16(const CUtensorMap &kmap, const CUtensorMap &vmap,
                                      const DecodeArgs &args, int head_dim, bool kv8, bool partial,
                                      int units, cudaStream_t stream);
// The many-row kernel, single pass, writing its rows' statistics (row_nlse).
cudaError_t launch_prefill_stats(const CUtensorMap &kmap, const CUtensorMap &vmap,
                                 const CUtensorMap &qmap, const DecodeArgs &args, int head_dim,
                                 bool fp16, bool kv8, cudaStream_t stream);

}  // namespace pa
