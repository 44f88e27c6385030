// Backward of the weighted expert-major combine out[t] = sum_j w[t, j] y[row(t, j)]:
//   grad_y[row(t, j)] = w[t, j] grad_out[t]            (bf16, or e4m3 with a scale per 128 channels)
//   grad_w[t, j]      = sum_h grad_out[t, h] y[row(t, j), h]
//
// HBM-bound: an entry's row of y is read once and its row of grad_y written
// once; the token's row of grad_out serves its k entries from L1 and L2.  A warp
// takes an entry, so the entries of a token are neighbours in a block, and the dot
// product ends in one exchange inside the warp: its order, and with it the result,
// is always the same.
#include "device_common.cuh"
#include "ep_internal.h"
#include "experts.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBatch = 4;  // 16-byte words of a row that a lane has in flight

__device__ __forceinline__ uint4 ld_cached(const void* p) {
  uint4 v;
  asm("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

}  // namespace

template <bool kFP8>
__global__ void __launch_bounds__(kThreads, 4) k_combine_backward(const CombineBackwardArgs a) {
  const int lane = threadIdx.x & 31;
  const int words = a.H >> 3;
  for (long long i = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < a.entries;
       i += static_cast<long long>(gridDim.x) * kWarps) {
    const int e = a.ent_idx[i], slot = a.ent_slot[i];
    long long row = e >= 0 && slot >= 0 ? static_cast<long long>(a.expert_offset[e]) + slot : -1;
    if (row >= a.rows) {
      if (lane == 0) latch_error(a.err, kErrCapacity);
      row = -1;
    }
    if (row < 0) {
      if (a.grad_weights && lane == 0) a.grad_weights[i] = 0.0f;
      continue;
    }
    const float w = a.topk_weights ? a.topk_weights[i] : 0.0f;
    const uint16_t* g = a.grad_out + i / a.k * a.H;
    const uint16_t* y = a.grad_weights ? a.y + row * a.H : nullptr;
    float dot = 0.0f;
    for (int c0 = lane; c0 - lane < words; c0 += 32 * kBatch) {
      uint4 gv[kBatch], yv[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int c = c0 + 32 * b;
        gv[b] = c < words ? ld_cached(g + 8 * c) : make_uint4(0, 0, 0, 0);
        if (y) yv[b] = c < words ? ld_stream(y + 8 * c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int c = c0 + 32 * b;
        const uint32_t gw[4] = {gv[b].x, gv[b].y, gv[b].z, gv[b].w};
        if (y) {
          const uint32_t yw[4] = {yv[b].x, yv[b].y, yv[b].z, yv[b].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dot = fmaf(bf16_lo(gw[j]), bf16_lo(yw[j]), dot);
            dot = fmaf(bf16_hi(gw[j]), bf16_hi(yw[j]), dot);
          }
        }
        if (a.grad_y) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[2 * j] = w * bf16_lo(gw[j]), v[2 * j + 1] = w * bf16_hi(gw[j]);
          if constexpr (kFP8) {
            // sixteen lanes hold a group of 128 channels
            float most = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(v[j]));
#pragma unroll
            for (int d = 8; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(kFullMask, most, d));
            float inv;
            const float sc = group_scale(most, &inv);
            if (c < words) {
              uint2 q = make_uint2(quant4(v, inv), quant4(v + 4, inv));
              *reinterpret_cast<uint2*>(static_cast<unsigned char*>(a.grad_y) + row * a.H + 8 * c) = q;
              if ((lane & 15) == 0) st_keep(a.grad_y_scales + (c >> 4) * a.scales_ld + row, sc);
            }
          } else if (c < words) {
            st_na(static_cast<uint16_t*>(a.grad_y) + row * a.H + 8 * c,
                  make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7])));
          }
        }
      }
    }
    if (a.grad_weights) {
#pragma unroll
      for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(kFullMask, dot, d);
      if (lane == 0) a.grad_weights[i] = dot;
    }
  }
}

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, bool fp8, int sms, cudaStream_t stream) {
  auto kernel = fp8 ? k_combine_backward<true> : k_combine_backward<false>;
  const long long need = (a.entries + kWarps - 1) / kWarps, most = static_cast<long long>(sms) * 4;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(kThreads), 0, stream, a);
}

}  // namespace ep
