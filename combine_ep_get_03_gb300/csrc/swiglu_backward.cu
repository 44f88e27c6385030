// Backward of the experts' activation from its 8-bit checkpoint.
//
// For a live row r with gate g and up u (dequantised e4m3), s = 1/(1+exp(-g)),
// routing weight w and incoming gradient d:
//   dg = d w u s (1 + g (1 - s)),  du = d w g s,  dw = sum_f d g s u.
// (dg, du) leave as e4m3 with a scale for every 128 channels, ready for the
// two products of the backward pass.
//
// One pass, bound by memory: 2 + 2 bytes read and 2 written for every channel.
// A warp owns a row, eight lanes a 128-channel group (16 channels a lane, 16-
// and 32-byte accesses), so the group maxima are three shuffles and dw stays
// in registers until the row ends: no atomics, the sum's order is fixed.
#include "ep_internal.h"
#include "experts.cuh"

namespace ep {

constexpr int kSwigluBackwardThreads = 256;

__global__ void __launch_bounds__(kSwigluBackwardThreads, 3) k_swiglu_backward(const SwigluBackwardArgs p) {
  extern __shared__ unsigned prefix[];
  __shared__ unsigned sums[32];
  groups_prefix(p.groups, 1, prefix, sums);
  const int lane = threadIdx.x & 31;
  const unsigned total = prefix[p.groups.G];
  const int F = p.F, Gf = F >> 7;
  const unsigned step = gridDim.x * (kSwigluBackwardThreads / 32);
  for (unsigned i = blockIdx.x * (kSwigluBackwardThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
    const int g = find_group(prefix, p.groups.G, i);
    long long start;
    const int n = group_span(p.groups, g, &start, false);
    const unsigned slot = i - prefix[g];
    if (slot >= static_cast<unsigned>(n)) continue;
    const long long row = start + slot;
    const float w = p.row_weights ? p.row_weights[row] : 1.0f;
    float dw = 0.0f;
    for (int f0 = 0; f0 < F; f0 += 512) {
      const int f = f0 + lane * 16;
      const bool on = f < F;  // whole groups of eight lanes
      float dg[16], du[16];
      float ag = 0.0f, au = 0.0f;
      if (on) {
        const unsigned char* pg = p.pre.data + row * (2LL * F) + f;
        const uint4 qg = ld_stream(pg), qu = ld_stream(pg + F);
        const uint16_t* pd = p.grad_act + row * F + f;
        const uint4 d0 = ld_stream(pd), d1 = ld_stream(pd + 8);
        const float sg = *p.pre.scale(row, f >> 7), su = *p.pre.scale(row, Gf + (f >> 7));
        const uint32_t wg[4] = {qg.x, qg.y, qg.z, qg.w}, wu[4] = {qu.x, qu.y, qu.z, qu.w};
        const uint32_t wd[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e4m3x4_to_f32(wg[j], dg + 4 * j);
          e4m3x4_to_f32(wu[j], du + 4 * j);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float gate = dg[j] * sg, up = du[j] * su;
          const float d = (j & 1) ? bf16_hi(wd[j >> 1]) : bf16_lo(wd[j >> 1]);
          const float s = __fdividef(1.0f, 1.0f + __expf(-gate));
          const float silu = gate * s;
          du[j] = d * silu;
          dw = fmaf(du[j], up, dw);
          // s (1 + g (1 - s)) = s (1 + g - silu)
          dg[j] = d * up * (s * (1.0f + gate - silu));
          ag = fmaxf(ag, fabsf(dg[j]));
          au = fmaxf(au, fabsf(du[j]));
        }
      }
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        ag = fmaxf(ag, __shfl_xor_sync(kFullMask, ag, d));
        au = fmaxf(au, __shfl_xor_sync(kFullMask, au, d));
      }
      if (on) {
        float ig, iu;
        // the row's weight multiplies the group's largest and the inverse scale
        const float sg = group_scale(ag * fabsf(w), &ig), su = group_scale(au * fabsf(w), &iu);
        ig *= w;
        iu *= w;
        unsigned char* q = p.grad_pre.data + row * (2LL * F) + f;
        *reinterpret_cast<uint4*>(q) = make_uint4(quant4(dg, ig), quant4(dg + 4, ig), quant4(dg + 8, ig), quant4(dg + 12, ig));
        *reinterpret_cast<uint4*>(q + F) = make_uint4(quant4(du, iu), quant4(du + 4, iu), quant4(du + 8, iu), quant4(du + 12, iu));
        if ((lane & 7) == 0) {
          *p.grad_pre.scale(row, f >> 7) = sg;
          *p.grad_pre.scale(row, Gf + (f >> 7)) = su;
        }
      }
    }
    if (p.grad_row_weights) {
#pragma unroll
      for (int d = 16; d; d >>= 1) dw += __shfl_xor_sync(kFullMask, dw, d);
      if (lane == 0) p.grad_row_weights[row] = dw;
    }
  }
}

cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& p, int sms, cudaStream_t stream) {
  const long long need = (p.groups.rows + kSwigluBackwardThreads / 32 - 1) / (kSwigluBackwardThreads / 32);
  const long long most = 3LL * sms;
  const unsigned blocks = static_cast<unsigned>(need < most ? (need > 0 ? need : 1) : most);
  return launch_kernel(k_swiglu_backward, dim3(blocks), dim3(kSwigluBackwardThreads),
                       sizeof(unsigned) * (p.groups.G + 1), stream, p);
}

}  // namespace ep
