// Log-probabilities, entropy and alternatives of rows of logits (logits.cu), as
// the transformer's forward calls them.
#pragma once

#include "../../include/mlora_logits.h"
#include "internal.h"

namespace mlk {

struct LogitsView {
    const void* x;
    int64_t ld;
    int64_t n_rows;
    const int* targets;                // null: none
    // row r's results go to row out_row[r] of the outputs, r's own where it is null.  With
    // it, rows r >= 128 row_tiles[0] - row0 and rows with out_row < 0 or a target < 0 are left out.
    const int* out_row;
    const int* row_tiles;
    int64_t row0;                      // the first row's number among those that row_tiles counts
    int* status;
    float scale;
    int V, dtype, top;
};

cudaError_t launch_token_logprobs(const LogitsView& x, const mlora_token_stats& out, int num_sms, cudaStream_t s);

// Checks of scale, top and vocabulary that the entry points share.
int logits_check(float scale, int32_t top, int32_t vocab);

}  // namespace mlk
