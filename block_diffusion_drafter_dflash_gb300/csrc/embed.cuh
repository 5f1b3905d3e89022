// Token embedding with a factor, and its gradient (embed.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dflash {

struct EmbedArgs {
  const void* table;        // [vocab][dim]
  const int32_t* tokens;    // [n]
  int n, vocab, dim;
  float scale;
  void* out;                // [n] rows of dim, out_stride elements apart
  int64_t out_stride;
};

// Scratch of a gradient call, carved from the caller's workspace.
struct EmbedBwdPlan {
  int n, vocab, dim;
  int pitch;                // values between the chunks' sums
  int chunks;               // of kEmbedChunk sorted tokens
  int32_t* kept;            // tokens inside the vocabulary
  uint2* order;             // [n] (token, position), sorted
  uint2* spare;             // [n] between the passes
  float* part;              // [chunks][2][pitch] sums of a chunk's first and last token where they go on outside
  size_t bytes;
};
constexpr int kEmbedChunk = 32;

struct EmbedBwdArgs {
  const void* d_out;        // [n] rows of dim, stride elements apart
  int64_t stride;
  const int32_t* tokens;
  float scale;
  void* d_table;            // [vocab][dim]
  int accumulate;
};

EmbedBwdPlan embed_bwd_plan(void* ws, int n, int dim, int vocab);
// Shared-memory opt-in of the sort (once per device).
cudaError_t embed_backward_prepare();
cudaError_t embed_launch(const EmbedArgs& a, bool table_f32, bool out_f32, int sms, cudaStream_t s);
cudaError_t embed_backward_launch(const EmbedBwdPlan& pl, const EmbedBwdArgs& a, bool out_f32, bool table_f32, int sms,
                                  int* launches, cudaStream_t s);

}  // namespace dflash
