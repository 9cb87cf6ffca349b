// Operators on tokens and rows of logits: sampling, the largest logits of a row, and the
// embedding with its gradient.  The calls' arguments as the kernels take them, and the host
// launchers.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dspark {

constexpr int kMaxTop = 1024;        // k of dspark_top_logits, at most

// Rows of logits; either `tokens` (a draw) or `ids` (the k largest) is given.
struct RowArgs {
  int T, V, dtype;
  long long ld;                      // elements from a row to the next
  const void* logits;
  // a draw: the settings, each for every row unless an array brings a row's own
  float temperature, top_p, min_p;
  int top_k;
  const float *row_temperature, *row_top_p, *row_min_p;
  const int32_t* row_top_k;
  const float* uniform;
  int32_t* tokens;
  float* logp;
  bool long_first;                   // (of the launch: two CTAs a row, see k_sample.cu)
  // the largest
  int k;
  int32_t* ids;
  float *values, *lse;
  cudaStream_t stream;
};

cudaError_t launch_rows(const RowArgs& a);           // k_sample.cu

struct EmbedArgs {
  int T, V, H, dtype;
  float scale;
  const int32_t* ids;
  const void *table, *d_out, *add;   // add: NULL, or what the gradient is added to
  void *out, *d_table;
  // the gradient's workspace
  uint32_t* ctrl;
  uint32_t *key[2], *pos[2];         // [T] (token, row) pairs while and after they are sorted
  uint32_t* hist;                    // [bins][tiles] digit counts of the tiles of a sort
  uint8_t* there;                    // [V] behind ctrl's 256 bytes: 1 for a token that occurs
  float* part;                       // [chunks][2][H] sums of tokens that chunks share
  int32_t* part_tok;                 // [chunks][2] their tokens, -1: none
  int bits, chunk, chunks;
  cudaStream_t stream;
};

void plan_embed(EmbedArgs* a);                       // bits, chunk, chunks from T, V, H
size_t embed_hist_words(const EmbedArgs& a);
cudaError_t launch_embed(const EmbedArgs& a);                  // k_embed.cu
cudaError_t launch_embed_backward(const EmbedArgs& a);

}  // namespace dspark
