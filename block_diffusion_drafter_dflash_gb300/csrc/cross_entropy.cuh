// Softmax cross-entropy of hidden states against an LM head without keeping the
// logits, and its gradient (cross_entropy.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dflash {

// Shapes and scratch of one call, carved from the caller's workspace.  Rows are
// those whose target lies inside the vocabulary, in their order.
struct CePlan {
  int rows, dim, vocab;
  int planes;            // bf16 planes of an operand: 1 (bf16 tensors) or 3 (fp32 tensors)
  int direct;            // gradient: the hidden states' gradient needs no sums in memory
  int ctas, tile, bn;    // CTAs that share a tile, its rows and columns
  int rows_pad, dim_pad; // multiples of a tile's rows (256 for a pair of CTAs, else 128) and of 64
  int piece;             // vocabulary columns of a piece (a multiple of 256)
  int32_t* status;
  int32_t* kept;         // [2] rows kept; parts of a cut tile (the hidden states' gradient)
  int32_t* row_of;       // [rows_pad] the caller's row
  int32_t* target;       // [rows_pad]
  __nv_bfloat16* h;      // [planes][rows_pad][dim_pad]; zero behind the dim and the last kept row's tile
  float2* part;          // forward: [parts][rows_pad] (maximum, sum) of each half tile of columns
  float* picked;         // forward: [rows_pad] the target's exponent
  float2* lse2;          // gradient: [rows_pad] lse log2(e) as a rounded value and its residual
  float* gain;           // gradient: [rows_pad] d_loss / T
  float* rest;           // gradient: [rows_pad] what G's rounding leaves of the target's value (bf16 tensors)
  __nv_bfloat16* g;      // gradient: [planes][rows_pad][piece] gradient of a piece of the logits
  float* acc;            // gradient: [rows_pad][dim_pad] sums of the hidden states' gradient
  float* tail;           // gradient: sums of the parts of its tiles that are cut
  size_t bytes;
};

struct CeTensors {
  const void* hidden;
  int64_t row_stride;
  const void* weight;
  const int32_t* targets;
  float temperature;
  float *loss, *lse;                // forward
  const float *lse_in, *d_loss;     // gradient
  void* d_hidden;
  int64_t d_row_stride;
  void* d_weight;
};

// backward: the gradient's; want_hidden: with room for the sums of the hidden states' gradient
CePlan ce_plan(void* ws, int rows, int dim, int vocab, bool f32, bool backward, bool want_hidden, int sms);
// Shared-memory opt-in of the kernels (once per device).
cudaError_t ce_prepare_f32();
cudaError_t ce_prepare_bf16();
cudaError_t ce_forward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s);
cudaError_t ce_backward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s);

}  // namespace dflash
