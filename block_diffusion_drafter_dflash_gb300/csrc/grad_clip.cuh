// Global norm over many gradient tensors, and clipping by it (grad_clip.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dflash {

struct ClipTensor {
  const void* in;
  void* out;        // may be in
  int64_t numel;
  int bf16;         // 0: fp32
};

// CTAs of a launch, each with one partial sum (double) in the workspace.
int clip_grid(int sms);
size_t clip_workspace_bytes(int sms);

// norm[0] = sqrt(sum of squares over all tensors); where it is finite and
// above max_norm, out = in * (max_norm / norm), else out = in.
cudaError_t clip_grad_norm_launch(const ClipTensor* t, int n, float max_norm, float* norm, void* ws, int sms,
                                  int* launches, cudaStream_t s);

}  // namespace dflash
