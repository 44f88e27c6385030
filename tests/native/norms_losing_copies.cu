// The norms' kernels as they are, but with every thread but each block's first told
// that the copies it waited for never came, which they did: nothing is skipped.
#include "experts.cuh"

namespace ep {

__device__ __forceinline__ bool wait_and_lose(uint64_t* bar, uint32_t parity, volatile int* quit, int* err) {
  return wait_or_quit(bar, parity, quit, err) && threadIdx.x == 0;
}

}  // namespace ep

#define wait_or_quit wait_and_lose
#include "block_norm.cu"

extern "C" int lossy_forward(int T, int H, int res32, const void* post, const void* pre, const void* residual,
                             const void* y, void* new_residual, void* x, float* rstd, int sms, void* stream) {
  const ep::BlockNormArgs a{T, H, 1e-6f, 1.0f, 1, 0, post, pre, nullptr, nullptr, residual, y, new_residual, x, rstd};
  return ep::launch_block_norm(a, res32, sms, static_cast<cudaStream_t>(stream));
}

extern "C" int lossy_backward(int T, int H, int res32, const void* post, const void* pre, void* new_residual,
                              const void* y, float* rstd, const void* grad_new, const void* grad_x, void* grad_residual,
                              void* grad_y, float* grad_post, float* grad_pre, float* workspace, int sms, void* stream) {
  ep::BlockNormBackwardArgs a{};
  a.n = ep::BlockNormArgs{T, H, 0.0f, 1.0f, 1, 0, post, pre, nullptr, nullptr, nullptr, y, new_residual, nullptr, rstd};
  a.grad_new = grad_new;
  a.grad_x = grad_x;
  a.grad_residual = grad_residual;
  a.grad_y = grad_y;
  a.grad_post = grad_post;
  a.grad_pre = grad_pre;
  a.partial = workspace;
  return ep::launch_block_norm_backward(a, res32, sms, static_cast<cudaStream_t>(stream));
}
