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
// in registers until the row ends: no atomics, the sum's order is fixed.  The
// arithmetic (an exponential, a reciprocal, two quantisations) nearly fills the
// issue slots too, hence two channels an instruction where there is one.
// 32 768 rows of 2 048: 80 us, 5.1 TB/s; seven blocks of four warps per SM (28
// warps of 72 registers) against 86 us with three of eight warps, 97 us with
// one of sixteen; loading the next 512 channels while these compute: no gain.
#include "ep_internal.h"
#include "experts.cuh"

namespace ep {

constexpr int kSwigluBackwardThreads = 128;

namespace {

// Two fp32 operations an instruction: the kernel is bound by issue before
// memory, at 28 instructions a channel (counted on the device).
__device__ __forceinline__ uint64_t bits(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 pair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(r);
}
// 2^x and 1/x to about one part in 2^22
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Sixteen products x * inv as e4m3 codes.
__device__ __forceinline__ uint4 quant16(const float2* x, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = mul2(x[2 * j], make_float2(inv, inv)), b = mul2(x[2 * j + 1], make_float2(inv, inv));
    w[j] = pack_e4m3x2(a.x, a.y) | (pack_e4m3x2(b.x, b.y) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace

__global__ void __launch_bounds__(kSwigluBackwardThreads, 7) k_swiglu_backward(const SwigluBackwardArgs p) {
  extern __shared__ unsigned prefix[];
  __shared__ unsigned sums[32];
  after_previous();
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
    float2 dw = make_float2(0.0f, 0.0f);
    for (int f0 = 0; f0 < F; f0 += 512) {
      const int f = f0 + lane * 16;
      const bool on = f < F;  // whole groups of eight lanes
      float2 dg[8], du[8];
      float ag = 0.0f, au = 0.0f;
      if (on) {
        const unsigned char* pg = p.pre.data + row * (2LL * F) + f;
        const uint4 qg = ld_stream(pg), qu = ld_stream(pg + F);
        const uint16_t* pd = p.grad_act + row * F + f;
        const uint4 d0 = ld_stream(pd), d1 = ld_stream(pd + 8);
        const float sg = *p.pre.scale(row, f >> 7), su = *p.pre.scale(row, Gf + (f >> 7));
        const uint32_t wg[4] = {qg.x, qg.y, qg.z, qg.w}, wu[4] = {qu.x, qu.y, qu.z, qu.w};
        const uint32_t wd[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
        constexpr float kLog2e = 1.44269504088896341f;
        const float2 sg2 = make_float2(sg, sg), su2 = make_float2(su, su);
        const float2 arg2 = make_float2(-sg * kLog2e, -sg * kLog2e);
        const float2 one = make_float2(1.0f, 1.0f), minus = make_float2(-1.0f, -1.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e4m3x4_to_f32(wg[j], &dg[2 * j].x);
          e4m3x4_to_f32(wu[j], &du[2 * j].x);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 gate = mul2(dg[j], sg2), up = mul2(du[j], su2), t = mul2(dg[j], arg2);
          const float2 d = make_float2(bf16_lo(wd[j]), bf16_hi(wd[j]));
          const float2 e = add2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), one);
          const float2 s = make_float2(rcp_fast(e.x), rcp_fast(e.y));
          const float2 silu = mul2(gate, s);
          du[j] = mul2(d, silu);
          dw = fma2(du[j], up, dw);
          // s (1 + g (1 - s)): beyond g = 17 s is 1, so the product is 0 however large g is
          // (1 + g - silu would be 0 from 2^24 on)
          dg[j] = mul2(mul2(d, mul2(up, s)), fma2(gate, fma2(s, minus, one), one));
          ag = fmaxf(ag, fmaxf(fabsf(dg[j].x), fabsf(dg[j].y)));
          au = fmaxf(au, fmaxf(fabsf(du[j].x), fabsf(du[j].y)));
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
        st_na(q, quant16(dg, ig));
        st_na(q + F, quant16(du, iu));
        if ((lane & 7) == 0) {
          *p.grad_pre.scale(row, f >> 7) = sg;
          *p.grad_pre.scale(row, Gf + (f >> 7)) = su;
        }
      }
    }
    if (p.grad_row_weights) {
      dw.x += dw.y;
#pragma unroll
      for (int d = 16; d; d >>= 1) dw.x += __shfl_xor_sync(kFullMask, dw.x, d);
      if (lane == 0) p.grad_row_weights[row] = dw.x;
    }
  }
}

cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& p, int sms, cudaStream_t stream) {
  const long long need = (p.groups.rows + kSwigluBackwardThreads / 32 - 1) / (kSwigluBackwardThreads / 32);
  const long long most = 7LL * sms;
  const unsigned blocks = static_cast<unsigned>(need < most ? (need > 0 ? need : 1) : most);
  return launch_kernel(k_swiglu_backward, dim3(blocks), dim3(kSwigluBackwardThreads),
                       sizeof(unsigned) * (p.groups.G + 1), stream, p);
}

}  // namespace ep
