// Kernels of the transformer model's rollouts besides the cache operators.
#pragma once

#include "kv_common.cuh"

namespace mlk {

// Positions of a rollout batch's padded rows from its sequences (rows without
// one: position 0 and target -1, ranges raised), and in row_map the padded row
// of each of the n batch rows; a row with a bad adapter id has none and gets row
// max_rows - 1, which no tile holds: at most n - 1 rows are routed then, and
// max_rows is the row bound of n.
void launch_tf_cached_rows(const KvView& c, const int* perm_pad, const int* meta, const int* inv, int n,
                           int max_rows, int* pos_pad, int* tgt_pad, int* row_map, int* status, cudaStream_t s);

// The last rows of the sequences, out of xf (padded rows), side by side in x:
// perm[s] = s and tgt[s] = 0 for a sequence with a good one, -1 for the others
// and for the rows that fill the last 128; meta[0] the row tiles.
void launch_tf_last_rows(const KvView& c, const int* inv, const int* tgt_pad, const bf16* xf, int d,
                         bf16* x, int* perm, int* tgt, int* meta, cudaStream_t s);

// Next tokens (sampling.cuh) of the n rows of x from their partials and lse.
void launch_tf_sample(const float* part, int n_nt, int part_ld, const float* lse, const int* perm, const bf16* x,
                      const bf16* Wout, int d, int V, const float* uniforms, int n, int* next_out, float* logprob_out,
                      int* status, cudaStream_t s);

}  // namespace mlk
