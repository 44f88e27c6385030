// One value per expert-major row back to the (token, k) entry it belongs to:
// the combine of recv_weights' gradients.  A gather of one word per entry; the
// rows' words and the entries' expert and slot are read once, coalesced on the
// entries' side.
#include "ep_internal.h"
#include "experts.cuh"

namespace ep {

__global__ void k_em_combine_weights(const int* idx, const int* slot, const int* offset, const float* row_weights,
                                     long long rows, long long entries, float* out, int* err) {
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= entries) return;
  float v = 0.0f;
  const int e = idx[i];
  if (e >= 0) {
    const long long row = static_cast<long long>(offset[e]) + slot[i];
    if (row < rows)
      v = row_weights[row];
    else
      latch_error(err, kErrCapacity);
  }
  out[i] = v;
}

cudaError_t launch_em_combine_weights(const int* idx, const int* slot, const int* offset, const float* row_weights,
                                      long long rows, long long entries, float* out, int* err, cudaStream_t stream) {
  return launch_kernel(k_em_combine_weights, dim3(static_cast<unsigned>((entries + 255) / 256)), dim3(256), 0, stream,
                       idx, slot, offset, row_weights, rows, entries, out, err);
}

}  // namespace ep
