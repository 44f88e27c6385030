// Weighted combine of expert-major rows: out[t] = bf16( sum over t's unmasked
// entries, ascending expert id (k-index breaks ties), of w[t, j] y[row(t, j)] ), a
// fused multiply-add in fp32 for each, from +0.0.
//
// HBM-bound gather: every row is read once, out written once.  A warp takes 1024
// channels of a token, 512 at a time, and asks for all sources of such a slab (up to
// eight) before it adds the first, so that it has up to 8 KB in flight; L2 is told of
// the rest of the 1024 meanwhile.  Two blocks of eight warps an SM, items dealt
// round.  8 192 tokens of 8 rows, 7168 channels: 154 us, 6.75 TB/s.
#include <climits>

#include "device_common.cuh"
#include "em_combine.cuh"
#include "ep_internal.h"
#include "pairs.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSlab = 512, kPart = 2 * kSlab;  // channels
constexpr int kSources = 8;                    // rows asked for together

}  // namespace

__global__ void __launch_bounds__(kThreads, 2) k_combine_weighted(const CombineWeightedArgs a) {
  // a token's rows and weights in the order of their sum
  __shared__ long long rows_of[kWarps][32];
  __shared__ float weights_of[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const EmEntries& n = a.entries;
  const int parts = (a.H + kPart - 1) / kPart;
  const long long items = static_cast<long long>(n.T) * parts;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long item = static_cast<long long>(blockIdx.x) * kWarps + warp; item < items; item += step) {
    const long long t = item / parts;
    const int begin = static_cast<int>(item - t * parts) * kPart, end = min(a.H, begin + kPart);
    long long row = -1;
    float w = 0.0f;
    int key = INT_MAX;
    if (lane < n.k) {
      const int e = n.idx[t * n.k + lane], slot = n.slot[t * n.k + lane];
      if (e >= 0 && slot >= 0) {
        row = static_cast<long long>(n.offset[e]) + slot;
        w = a.topk_weights[t * n.k + lane];
        key = e;
      }
      if (row >= a.rows) {
        latch_error(n.err, kErrCapacity);
        row = -1;
        key = INT_MAX;
      }
    }
    const int sources = __popc(__ballot_sync(kFullMask, row >= 0));
    int place = 0;
    for (int j = 0; j < n.k; ++j) {
      const int other = __shfl_sync(kFullMask, key, j);
      place += other < key || (other == key && j < lane);
    }
    if (row >= 0) {
      rows_of[warp][place] = row;
      weights_of[warp][place] = w;
      if (begin + kSlab < end)
        prefetch_l2_bulk(a.y + row * a.H + begin + kSlab, static_cast<uint32_t>(end - begin - kSlab) * 2);
    }
    __syncwarp();
    for (int h = begin + 8 * lane; h - 8 * lane < end; h += kSlab) {
      const bool on[2] = {h < end, h + kSlab / 2 < end};
      float2 sum[2][4];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[c][i] = both(0.0f);
      for (int s0 = 0; s0 < sources; s0 += kSources) {
        uint4 v[kSources][2];
#pragma unroll
        for (int s = 0; s < kSources; ++s) {
          if (s0 + s >= sources) continue;
          const uint16_t* y = a.y + rows_of[warp][s0 + s] * a.H + h;
#pragma unroll
          for (int c = 0; c < 2; ++c) v[s][c] = on[c] ? ld_stream(y + c * (kSlab / 2)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < kSources; ++s) {
          if (s0 + s >= sources) continue;
          const float2 by = both(weights_of[warp][s0 + s]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t q[4] = {v[s][c].x, v[s][c].y, v[s][c].z, v[s][c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[c][i] = fma2(by, make_float2(bf16_lo(q[i]), bf16_hi(q[i])), sum[c][i]);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (on[c])
          st_na(a.out + t * a.H + h + c * (kSlab / 2),
                make_uint4(pack_bf16x2(sum[c][0].x, sum[c][0].y), pack_bf16x2(sum[c][1].x, sum[c][1].y),
                           pack_bf16x2(sum[c][2].x, sum[c][2].y), pack_bf16x2(sum[c][3].x, sum[c][3].y)));
    }
    __syncwarp();  // read before the next item writes
  }
}

cudaError_t launch_combine_weighted(const CombineWeightedArgs& a, int sms, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.entries.T) * ((a.H + kPart - 1) / kPart);
  const long long need = (items + kWarps - 1) / kWarps, most = static_cast<long long>(sms) * 2;
  return launch_kernel(k_combine_weighted, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(kThreads), 0,
                       stream, a);
}

}  // namespace ep
