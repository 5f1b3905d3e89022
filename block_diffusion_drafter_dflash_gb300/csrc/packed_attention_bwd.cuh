// Gradients of the packed training attention (packed_attention_bwd.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dflash {

// Shapes and operand layout of one call, carved from the caller's workspace.
// Rows are the blocks in ascending order of their anchors, whole blocks to a
// tile of 128 rows (`per` of them, then padding).
struct PackedBwdPlan {
  int N, block, S, nq, nkv, hd;
  int planes;             // fp16 operand planes: 1 (bf16 tensors) or 2 (fp32 tensors as hi + lo)
  int per;                // blocks in a row tile
  int T;                  // row tiles
  int KT;                 // 128-key tiles of the context
  int share;              // streamed tiles that one CTA takes of a (kv head, context key tile)
  int splits;             // CTAs that may share one
  int parts;              // CTAs that look for the operands' ranges
  int32_t* status;
  float* part;            // [parts][kRangeValues] their maxima
  int32_t* scale;         // [5] exponents of the powers of two the operands are scaled by (Scales)
  int32_t* order;         // [N] block of each sorted place
  int32_t* sorted;        // [N] anchors in ascending order
  int2* seen_by;          // [KT] first row tile that sees some of the key tile, and all of it
  int32_t* row_anchor;    // [T*128] anchor of the row's block (INT_MAX in padding)
  float* lse2;            // [nq][T*128] lse log2(e) - kPExp, +inf in padding
  float* delta;           // [nq][T*128] sum_d d_out out, scaled as dp
  float* row_scale;       // [nq][T*128] power of two that the row's ds may be larger by in dQ
  __half* q;              // [nq][planes][T*128][hd], zero in padding (d_o, kb and vb too)
  __half* d_o;
  __half* kc;             // [nkv][planes][KT*128][hd]
  __half* vc;
  __half* kb;             // [nkv][planes][T*128][hd]
  __half* vb;
  float* dk_part;         // [nkv][splits][KT*128][hd] each share's sum of d_k_ctx
  float* dv_part;
  size_t bytes;
};

PackedBwdPlan packed_bwd_plan(void* ws, int N, int block, int S, int nq, int nkv, int hd, bool f32, int sms);

struct PackedBwdTensors {
  const void *q, *k_ctx, *v_ctx, *k_blk, *v_blk;
  const int32_t* anchors;
  const float *out, *lse, *d_out;
  void *d_q, *d_k_ctx, *d_v_ctx, *d_k_blk, *d_v_blk;
};

// Shared-memory opt-in of the gradient kernel (once per device).
cudaError_t packed_bwd_prepare(int hd, bool f32);
cudaError_t packed_bwd_run(const PackedBwdPlan& pl, const PackedBwdTensors& t, int sms, int* launches, cudaStream_t s);

// lse[n][i][h] = ln of the softmax denominator of each query row, from the
// forward's split partials.
cudaError_t packed_lse_launch(const float2* ml, int N, int block, int nq, int splits, float* lse, cudaStream_t s);

}  // namespace dflash
