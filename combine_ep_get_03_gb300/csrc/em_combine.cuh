// The weighted combine of expert-major rows and its gradient (combine_weighted.cu,
// combine_backward.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ep {

// The entries' places in the handle's last expert-major layout.
struct EmEntries {
  const int* idx;     // [T][k] expert, -1 masked
  const int* slot;    // [T][k] row inside the expert
  const int* offset;  // [E+1] first row of each expert
  int T, k;
  int* err;
};

struct CombineWeightedArgs {
  EmEntries entries;
  const uint16_t* y;          // [rows][H] bf16
  const float* topk_weights;  // [T][k]
  uint16_t* out;              // [T][H] bf16
  long long rows;
  int H;
};
cudaError_t launch_combine_weighted(const CombineWeightedArgs& a, int sms, cudaStream_t stream);

struct CombineBackwardArgs {
  EmEntries entries;
  const uint16_t* grad_out;    // [T][H] bf16
  const uint16_t* y;           // [rows][H] bf16 (with grad_weights)
  const float* topk_weights;   // [T][k] (with grad_y)
  void* grad_y;                // [rows][H] bf16 or e4m3, or null
  float* grad_y_scales;        // [H/128][scales_ld] (e4m3)
  float* grad_weights;         // [T][k] or null
  long long scales_ld, rows;
  int H;
};
cudaError_t launch_combine_backward(const CombineBackwardArgs& a, bool fp8, int sms, cudaStream_t stream);

}  // namespace ep
