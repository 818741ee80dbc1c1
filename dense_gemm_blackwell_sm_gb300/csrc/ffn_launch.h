// ffn_launch.h -- internal interface between the feed-forward block's C entry
// points (ffn.cu) and its kernel translation units.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ffn.h"

namespace dgb {

// What a launch needs to know about the current device.
struct FfnDevice {
  int num_sms;
  uint32_t* status;  // device status word of the bounded waits
};

// The current device, checked once to be one this library has code for; `word` 0: the
// feed-forward operators' status word, 1: that of quant.h's.
gemm_status_t device_of_call(int word, FfnDevice* out);
// synchronises the stream, then reports and clears that word
gemm_status_t check_word(int word, cudaStream_t st);

// raise a kernel's dynamic shared-memory limit, once per device
cudaError_t allow_smem_once(const void* func, size_t bytes);

// CTAs of a kernel an SM holds at once with `smem` bytes of dynamic shared memory (its
// limit is raised to `most`), asked once per device
cudaError_t resident_ctas(const void* func, int threads, size_t smem, size_t most, int* out);

// The pitches below are resolved (never 0).
cudaError_t launch_gated(const ffn_gated_t& a, const FfnDevice& dev, cudaStream_t st);
size_t gated_backward_workspace(const ffn_gated_grad_t& a);
cudaError_t launch_gated_backward(const ffn_gated_grad_t& a, const FfnDevice& dev, cudaStream_t st);

cudaError_t launch_norm(const ffn_norm_t& a, const FfnDevice& dev, cudaStream_t st);
size_t norm_backward_workspace(const ffn_norm_grad_t& a);
cudaError_t launch_norm_backward(const ffn_norm_grad_t& a, const FfnDevice& dev, cudaStream_t st);

}  // namespace dgb
