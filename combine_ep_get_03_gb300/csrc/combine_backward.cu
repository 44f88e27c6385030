// Backward of the weighted expert-major combine out[t] = sum_j w[t, j] y[row(t, j)]:
//   grad_y[row(t, j)] = w[t, j] grad_out[t]            (bf16, or e4m3 with a scale per 128 channels)
//   grad_w[t, j]      = sum_h grad_out[t, h] y[row(t, j), h]
//
// HBM-bound: an entry's row of y is read once and its row of grad_y written
// once; the token's row of grad_out serves its k entries from L1 and L2.  A warp
// takes an entry, so the entries of a token are neighbours in a block, and the dot
// product ends in one exchange inside the warp: its order, and with it the result,
// is always the same.  8 192 tokens of 8 rows, 7168 channels: bf16 rows 311 us (6.4
// TB/s), e4m3 240 (6.3); with each group's maximum and divisions in all of its lanes
// 301.  Bulk prefetches of the next entry's row to L2 made it 373.
#include "device_common.cuh"
#include "em_combine.cuh"
#include "ep_internal.h"
#include "experts.cuh"
#include "pairs.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBatch = 4;  // 16-byte words of a row that a lane has in flight

__device__ __forceinline__ uint4 ld_cached(const void* p) {
  uint4 v;
  asm("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The larger of two pairs of bf16; a NaN loses.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace

template <bool kFP8>
__global__ void __launch_bounds__(kThreads, 4) k_combine_backward(const CombineBackwardArgs a) {
  const int lane = threadIdx.x & 31;
  const int words = a.H >> 3;
  const EmEntries& n = a.entries;
  const long long entries = static_cast<long long>(n.T) * n.k;
  for (long long i = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < entries;
       i += static_cast<long long>(gridDim.x) * kWarps) {
    const int e = n.idx[i], slot = n.slot[i];
    long long row = e >= 0 && slot >= 0 ? static_cast<long long>(n.offset[e]) + slot : -1;
    if (row >= a.rows) {
      if (lane == 0) latch_error(n.err, kErrCapacity);
      row = -1;
    }
    if (row < 0) {
      if (a.grad_weights && lane == 0) a.grad_weights[i] = 0.0f;
      continue;
    }
    const float w = a.topk_weights ? a.topk_weights[i] : 0.0f;
    const uint16_t* g = a.grad_out + i / n.k * a.H;
    const uint16_t* y = a.grad_weights ? a.y + row * a.H : nullptr;
    float2 dot = both(0.0f);
    for (int c0 = lane; c0 - lane < words; c0 += 32 * kBatch) {
      uint4 gv[kBatch], yv[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int c = c0 + 32 * b;
        gv[b] = c < words ? ld_cached(g + 8 * c) : make_uint4(0, 0, 0, 0);
        if (y) yv[b] = c < words ? ld_stream(y + 8 * c) : make_uint4(0, 0, 0, 0);
      }
      float inv = 0.0f;
      if (kFP8 && a.grad_y) {
        // Sixteen lanes hold a group of 128 channels, and a batch four groups of
        // theirs: the maxima of |grad_out| are halved in number as they are exchanged, so that
        // lanes 4 n + b end with group b's.  The largest |w grad_out| is |w| times that.
        uint32_t m[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          m[b] = max2(max2(gv[b].x & 0x7fff7fffu, gv[b].y & 0x7fff7fffu), max2(gv[b].z & 0x7fff7fffu, gv[b].w & 0x7fff7fffu));
        const bool odd = lane & 1, upper = lane & 2;
        const uint32_t m01 = max2(odd ? m[1] : m[0], __shfl_xor_sync(kFullMask, odd ? m[0] : m[1], 1));
        const uint32_t m23 = max2(odd ? m[3] : m[2], __shfl_xor_sync(kFullMask, odd ? m[2] : m[3], 1));
        uint32_t most = max2(upper ? m23 : m01, __shfl_xor_sync(kFullMask, upper ? m01 : m23, 2));
        most = max2(most, __shfl_xor_sync(kFullMask, most, 4));
        most = max2(most, __shfl_xor_sync(kFullMask, most, 8));
        const float sc = group_scale(fabsf(w) * fmaxf(bf16_lo(most), bf16_hi(most)), &inv);
        const int c = c0 + 32 * (lane & 3);
        if ((lane & 12) == 0 && c < words) st_keep(a.grad_y_scales + (c >> 4) * a.scales_ld + row, sc);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int c = c0 + 32 * b;
        const uint32_t gw[4] = {gv[b].x, gv[b].y, gv[b].z, gv[b].w};
        const uint32_t yw[4] = {yv[b].x, yv[b].y, yv[b].z, yv[b].w};
        float2 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = make_float2(bf16_lo(gw[j]), bf16_hi(gw[j]));
          if (y) dot = fma2(v[j], make_float2(bf16_lo(yw[j]), bf16_hi(yw[j])), dot);
          v[j] = mul2(v[j], both(w));
        }
        if (!a.grad_y) continue;
        if constexpr (kFP8) {
          const float2 by = both(__shfl_sync(kFullMask, inv, (lane & 16) + b));
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], by);
          if (c < words)
            *reinterpret_cast<uint2*>(static_cast<unsigned char*>(a.grad_y) + row * a.H + 8 * c) =
                make_uint2(pack_e4m3x2(v[0].x, v[0].y) | (pack_e4m3x2(v[1].x, v[1].y) << 16),
                           pack_e4m3x2(v[2].x, v[2].y) | (pack_e4m3x2(v[3].x, v[3].y) << 16));
        } else if (c < words) {
          st_na(static_cast<uint16_t*>(a.grad_y) + row * a.H + 8 * c,
                make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                           pack_bf16x2(v[3].x, v[3].y)));
        }
      }
    }
    if (a.grad_weights) {
      float sum = dot.x + dot.y;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
      if (lane == 0) a.grad_weights[i] = sum;
    }
  }
}

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, bool fp8, int sms, cudaStream_t stream) {
  auto kernel = fp8 ? k_combine_backward<true> : k_combine_backward<false>;
  const long long entries = static_cast<long long>(a.entries.T) * a.entries.k, need = (entries + kWarps - 1) / kWarps;
  const long long most = static_cast<long long>(sms) * 4;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(kThreads), 0, stream, a);
}

}  // namespace ep
