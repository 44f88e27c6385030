// Arguments of the norms around a block (block_norm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ep {

constexpr int kBlockNormMaxBlocks = 256;  // blocks whose partial sums the workspace holds
constexpr int kBlockNormMaxHidden = 16384;

struct BlockNormArgs {
  int T, H;
  float eps, scale;
  int weight32, gate_per_token;
  const void* post;     // [H] or null
  const void* pre;      // [H] or null
  const void* gate;     // [H], or bf16 [T][H] per token, or null
  const uint8_t* mask;  // [T] or null: 0 = padding token
  const void* residual;  // [T][H]
  const void* y;         // bf16 [T][H] or null
  void* new_residual;    // [T][H]
  void* x;               // bf16 [T][H] or null
  float* rstd;           // [2][T] or null
};

struct BlockNormBackwardArgs {
  BlockNormArgs n;       // residual and x unused; new_residual, y and rstd are inputs
  const void* grad_new;  // [T][H] or null: 0
  const void* grad_x;    // bf16 [T][H] or null: no norm behind
  void* grad_residual;   // [T][H] or null
  void* grad_y;          // bf16 [T][H] or null
  void* grad_gate;       // fp32 [H], or bf16 [T][H] per token, or null
  float* grad_post;      // [H] or null
  float* grad_pre;       // [H] or null
  float* partial;        // [blocks][2][H]
  int need_y, sum_y;     // set by the launch: y is read; its sum over tokens is wanted
};

cudaError_t launch_block_norm(const BlockNormArgs& a, bool res32, int sms, cudaStream_t stream);
cudaError_t launch_block_norm_backward(const BlockNormBackwardArgs& a, bool res32, int sms, cudaStream_t stream);

}  // namespace ep
