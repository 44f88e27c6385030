// The gate: top-k choice of experts, their weights, per-expert counts and the
// balance loss; and the gradient of both with respect to the logits.
//
// Per token t with logits l (fp32 arithmetic whatever their type):
//   choice   the k largest logits (of the topk_groups groups with the largest
//            maxima), ties to the lower index; -inf and NaN are never chosen
//   softmax  w_j = exp(l_j) / sum_chosen exp(l),  p_e = exp(l_e) / sum_E exp(l)
//   sigmoid  s = 1/(1+exp(-l)), w_j = s_j / sum_chosen s, p_e = s_e / sum_E s
// and over the V unmasked tokens, with c_e entries of expert e:
//   P_e = sum_t p_te / V,   loss = coef E / (k V) sum_e c_e P_e.
// Backward (r_e = 1 for softmax, 1 - s_e for sigmoid):
//   dl_e  = dloss coef E / (k V^2) p_e r_e (c_e - sum_j p_j c_j)
//         + [e chosen] w_e r_e (dw_e - sum_chosen w dw).
//
// A warp owns a token and a lane VPL consecutive experts in registers, so a
// lane's experts are the same for every token and the column sums P stay in
// registers until the block ends; lane order is index order, which settles
// ties by the first lane of a ballot.  Blocks join their sums as 64-bit fixed
// point, which makes the result independent of their order, and the last block
// to finish writes counts, P and the loss: one launch.  A sum is at most T, so
// the step is 2^-(63 - ceil(log2 T)): 2^-48 at 32 768 tokens.
//
// No pipe is full: the half-rate integer and compare pipe is 60 % busy forward
// (hence keys sorted once per lane and shifted, one score kind per row, bf16
// logits' exact 32-bit keys), and each token begins with a load that it waits
// for.  32 768 tokens of 256 bf16 logits, top-8: 27 us forward,
// 22 us backward (46 us the pair in a stream); one token 6 us, less than the
// call's host side.
#include <math_constants.h>

#include "ep_internal.h"
#include "experts.cuh"

namespace ep {

// Warps of a block: as many as leave room for a row of floats each.  Beyond 1 024
// experts (VPL = 128) a row does not fit the registers (1.6-1.9 KB of spill stores
// a thread): fp32, 8 192 tokens, top-8, forward and backward 53 and 79 us at 1 024
// experts, 257 and 312 at 1 025, 513 and 379 at 4 096.
__host__ __device__ constexpr int gate_warps(int vpl) { return vpl <= 8 ? 16 : vpl <= 32 ? 8 : 1; }
__host__ __device__ constexpr int index_bits(int vpl) { return vpl == 1 ? 5 : 1 + index_bits(vpl / 2); }

// work: [0] finished blocks, [1] set if a row had no finite sum, [2] unmasked
// tokens, [3] unused, then E u64 sums, then E counts
__device__ __forceinline__ unsigned long long* work_sums(unsigned* w) {
  return reinterpret_cast<unsigned long long*>(w + 4);
}
__device__ __forceinline__ int* work_counts(unsigned* w, int E) { return reinterpret_cast<int*>(w + 4 + 2 * E); }

// Order-preserving image of a float that is not NaN, equal for -0 and +0.
// -inf has the image kNever; what is not above it is never chosen.
constexpr unsigned kNever = 0x007fffffu;
__device__ __forceinline__ unsigned order_key(float v) {
  const unsigned b = __float_as_uint(v + 0.0f);
  return b ^ (static_cast<unsigned>(static_cast<int>(b) >> 31) | 0x80000000u);
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// The lane's VPL logits of a row, -inf past E.
template <typename T, int VPL>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, bool vec, float* v) {
  constexpr int kChunk = 16 / sizeof(T);
  const int e0 = lane * VPL;
  if constexpr (VPL % kChunk == 0) {
    if (vec) {
#pragma unroll
      for (int j = 0; j < VPL; j += kChunk) {
        if (e0 + j < E) {
          const uint4 q = *reinterpret_cast<const uint4*>(row + e0 + j);
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            v[j + i] = sizeof(T) == 4 ? __uint_as_float(w[i & 3]) : (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        } else {
#pragma unroll
          for (int i = 0; i < kChunk; ++i) v[j + i] = -CUDART_INF_F;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) v[j] = e0 + j < E ? load_logit(row + e0 + j) : -CUDART_INF_F;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kFullMask, x, d);
  return x;
}
// s / all, exactly 1 where s is all there is (its gradient is then exactly 0).
__device__ __forceinline__ float share_of(float s, float all) { return s == all ? 1.0f : __fdividef(s, all); }

// Sum and largest over the first k lanes, for the lanes below the next power
// of two; lanes from k on hold 0 and -inf.
__device__ __forceinline__ float sum_first(float x, int k) {
  for (int d = 1; d < k; d <<= 1) x += __shfl_xor_sync(kFullMask, x, d);
  return x;
}
__device__ __forceinline__ float max_first(float x, int k) {
  for (int d = 1; d < k; d <<= 1) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, d));
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, d));
  return x;
}

// e^x to a few parts in 10^7 for the x that matter (an error of 2^-24 |x|).
__device__ __forceinline__ float exp_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504088896341f));
  return r;
}

// Unnormalised score of a logit v, and its slope d log(score) / dv:
//   softmax            e^(v - m), m the row's largest;              slope 1
//   sigmoid, m >= 0    1 / (1 + e^-v);                               slope 1 - sigmoid(v)
//   sigmoid, m < 0     e^(v - m) / (1 + e^v), which stays away from 0/0 when
//                      every sigmoid underflows;                     slope 1 - sigmoid(v)
// One kind holds for a row, so it is chosen once and the logits' arithmetic has
// no selection (the half-rate integer and compare pipe bounds these kernels).
enum ScoreKind { kSoftmax, kSigmoid, kSmallSigmoid };
__device__ __forceinline__ ScoreKind score_kind(float& m, int sigmoid) {
  if (m == -CUDART_INF_F) m = 0.0f;
  return !sigmoid ? kSoftmax : m < 0.0f ? kSmallSigmoid : kSigmoid;
}
template <ScoreKind kKind>
__device__ __forceinline__ float score_of(float v, float m, float* slope) {
  if (kKind == kSoftmax) {
    if (slope) *slope = 1.0f;
    return exp_of(v - m);
  }
  const float e = exp_of(kKind == kSigmoid ? -v : v);
  const float r = __fdividef(1.0f, 1.0f + e);  // 0 from e = 2^126 on
  if (kKind == kSigmoid) {
    if (slope) *slope = fminf(e, 3.0e38f) * r;
    return r;
  }
  if (slope) *slope = r;
  return exp_of(v - m) * r;
}
template <int N>
__device__ __forceinline__ void score_row(ScoreKind kind, const float* v, float m, float* x, float* slope) {
  if (kind == kSoftmax) {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = score_of<kSoftmax>(v[j], m, slope ? slope + j : nullptr);
  } else if (kind == kSigmoid) {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = score_of<kSigmoid>(v[j], m, slope ? slope + j : nullptr);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = score_of<kSmallSigmoid>(v[j], m, slope ? slope + j : nullptr);
  }
}

// The lane's values sorted out of the keys c[] (order keys whose low bits are
// replaced by the inverted index, 0 = never chosen): the largest of the warp.
template <int VPL>
__device__ __forceinline__ unsigned local_max(const unsigned* c) {
  unsigned m = c[0];
#pragma unroll
  for (int j = 1; j < VPL; ++j) m = max(m, c[j]);
  return m;
}

// A lane's keys in descending order (Batcher's merge exchange network), so
// that dropping the largest is a shift.
template <int VPL>
__device__ __forceinline__ void sort_down(unsigned* c) {
#pragma unroll
  for (int p = 1; p < VPL; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < VPL; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < VPL && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const unsigned a = c[i + j], b = c[i + j + k];
            c[i + j] = max(a, b);
            c[i + j + k] = min(a, b);
          }
}

template <typename T, int VPL>
__global__ void __launch_bounds__(gate_warps(VPL) * 32) k_gate_forward(const GateArgs p) {
  constexpr int kWarps = gate_warps(VPL);
  constexpr int kBits = index_bits(VPL);
  constexpr unsigned kIndex = (1u << kBits) - 1u;
  extern __shared__ __align__(16) float sm[];  // [warps][32 VPL] sums, [E] counts, [warps][groups] keys
  int* s_count = reinterpret_cast<int*>(sm + kWarps * 32 * VPL);
  unsigned* s_group = reinterpret_cast<unsigned*>(s_count + p.E) + (threadIdx.x >> 5) * p.groups;
  __shared__ int s_live, s_bad, s_last;
  __shared__ float s_part[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = p.E, k = p.k;
  for (int e = tid; e < E; e += blockDim.x) s_count[e] = 0;
  if (tid == 0) s_live = 0, s_bad = 0;
  after_previous();
  __syncthreads();

  float acc[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) acc[j] = 0.0f;
  int live = 0;
  bool bad = false;
  const int gs = E / p.groups;
  // lanes of a group, where every group is a power of two of whole lanes
  const int span = gs % VPL == 0 && ((gs / VPL) & (gs / VPL - 1)) == 0 && gs / VPL <= 32 ? gs / VPL : 0;
  for (int t = blockIdx.x * kWarps + warp; t < p.T; t += gridDim.x * kWarps) {
    int my_id = -1;
    float my_w = 0.0f;
    if (!p.mask || p.mask[t]) {
      ++live;
      float v[VPL];
      load_row<T, VPL>(static_cast<const T*>(p.logits) + t * p.ld, E, lane, p.vec, v);
      // probabilities over all experts
      float mine = v[0];
#pragma unroll
      for (int j = 1; j < VPL; ++j) mine = fmaxf(mine, v[j]);
      {
        float m = warp_max(mine);
        const ScoreKind kind = score_kind(m, p.sigmoid);
        float x[VPL], sum = 0.0f;
        score_row<VPL>(kind, v, m, x, nullptr);  // 0 past E, where v is -inf
#pragma unroll
        for (int j = 0; j < VPL; ++j) sum += x[j];
        sum = warp_sum(sum);
        if (!(sum < CUDART_INF_F)) {
          // a NaN, or an infinity under softmax: the sums are marked, and the
          // choice goes on without the NaNs
          bad = true;
          mine = -CUDART_INF_F;
#pragma unroll
          for (int j = 0; j < VPL; ++j) {
            v[j] = fmaxf(v[j], -CUDART_INF_F);
            mine = fmaxf(mine, v[j]);
          }
        }
        const float inv = sum > 0.0f ? __fdividef(1.0f, sum) : 0.0f;  // a row of -inf has no probability
#pragma unroll
        for (int j = 0; j < VPL; ++j) acc[j] = fmaf(x[j], inv, acc[j]);
      }
      // experts of groups that are not kept drop out of the choice
      bool allowed = true;  // the lane's experts, where groups are whole lanes
      if (p.groups > 1) {
        if (span) {
          for (int d = 1; d < span; d <<= 1) mine = fmaxf(mine, __shfl_xor_sync(kFullMask, mine, d));
          // 0: taken, past the last expert, or not the group's first lane
          unsigned key = (lane & (span - 1)) == 0 && lane * VPL < E ? order_key(mine) : 0u;
          allowed = false;
          for (int i = 0; i < p.keep; ++i) {
            const unsigned top = __reduce_max_sync(kFullMask, key);
            const int src = __ffs(__ballot_sync(kFullMask, key == top)) - 1;
            if (lane == src) key = 0u;
            if ((lane & ~(span - 1)) == src) allowed = true;
          }
        } else {
          for (int g = lane; g < p.groups; g += 32) s_group[g] = 0u;
          __syncwarp();
          int g = min(lane * VPL, E - 1) / gs, left = (g + 1) * gs - lane * VPL;
          unsigned best = 0u;
#pragma unroll
          for (int j = 0; j < VPL; ++j) {
            if (lane * VPL + j < E) {
              if (left == 0) {
                atomicMax(&s_group[g], best);
                best = 0u, ++g, left = gs;
              }
              best = max(best, order_key(v[j]));
              --left;
            }
          }
          if (lane * VPL < E) atomicMax(&s_group[g], best);
          __syncwarp();
          // lane l ranks groups 2l and 2l + 1; 0: taken or absent
          unsigned long long kept = 0ull;
          unsigned g0 = 2 * lane < p.groups ? max(s_group[2 * lane], 1u) : 0u;
          unsigned g1 = 2 * lane + 1 < p.groups ? max(s_group[2 * lane + 1], 1u) : 0u;
          for (int i = 0; i < p.keep; ++i) {
            const unsigned top = __reduce_max_sync(kFullMask, max(g0, g1));
            const int src = __ffs(__ballot_sync(kFullMask, max(g0, g1) == top)) - 1;
            const int id = __shfl_sync(kFullMask, 2 * lane + (g0 == top ? 0 : 1), src);
            kept |= 1ull << id;
            if (lane == src) {
              if (g0 == top) g0 = 0u; else g1 = 0u;
            }
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < VPL; ++j)
            if (!((kept >> (min(lane * VPL + j, E - 1) / gs)) & 1ull)) v[j] = -CUDART_INF_F;
        }
      }
      // The k largest, one after another.  A key's low bits give way to the
      // inverted index, so one warp maximum names the expert and the owner
      // drops it by comparing.  bf16 keys lose nothing; of fp32 keys 32 - kBits
      // bits stay, and rows where two of the first k + 1 agree in them (about
      // one in a hundred) are settled again below, on whole keys.
      unsigned c[VPL];
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        c[j] = (order_key(v[j]) & ~kIndex) | (kIndex - (lane * VPL + j));
      }
      constexpr bool kSorted = VPL <= 16;  // more keys cost more to sort than to search again
      if (kSorted) sort_down<VPL>(c);
      unsigned best = kSorted ? c[0] : local_max<VPL>(c), my_key = 0u;
      if (!allowed) best = 0u;
      constexpr int kMore = sizeof(T) == 4 ? 1 : 0;
      if (kSorted && k <= 8) {
        // after pick i at most 8 - i more are wanted: shorter shifts
#pragma unroll
        for (int i = 0; i < 8 + kMore; ++i) {
          if (i >= k + kMore) break;
          const unsigned top = __reduce_max_sync(kFullMask, best);
          if (top <= kNever) break;
          if (lane == i) my_key = top;
          const bool drop = best == top;
#pragma unroll
          for (int j = 0; j < VPL && j < 8 - i; ++j) c[j] = drop ? (j + 1 < VPL ? c[j + 1] : 0u) : c[j];
          best = allowed ? c[0] : 0u;
        }
      } else {
        for (int i = 0; i < k + kMore && i < 32; ++i) {
          const unsigned top = __reduce_max_sync(kFullMask, best);
          if (top <= kNever) break;
          if (lane == i) my_key = top;
          if (kSorted) {
            const bool drop = best == top;
#pragma unroll
            for (int j = 0; j + 1 < VPL; ++j) c[j] = drop ? c[j + 1] : c[j];
            c[VPL - 1] = drop ? 0u : c[VPL - 1];
            best = allowed ? c[0] : 0u;
          } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j) c[j] = c[j] == top ? 0u : c[j];
            best = allowed ? local_max<VPL>(c) : 0u;
          }
        }
      }
      bool again = false;
      if (kMore) {
        const unsigned next = __shfl_down_sync(kFullMask, my_key, 1);
        again = k >= 32 || __any_sync(kFullMask, lane < k && my_key && next && ((my_key ^ next) & ~kIndex) == 0u);
      }
      if (!again) {
        if (lane < k && my_key) my_id = static_cast<int>(kIndex - (my_key & kIndex));
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) c[j] = allowed ? order_key(v[j]) : 0u;
        for (int i = 0; i < k; ++i) {
          best = local_max<VPL>(c);
          const unsigned top = __reduce_max_sync(kFullMask, best);
          if (top <= kNever) break;
          const int src = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
          int at = 0;
#pragma unroll
          for (int j = VPL - 1; j >= 0; --j)
            if (c[j] == top) at = j;
#pragma unroll
          for (int j = 0; j < VPL; ++j)
            if (lane == src && j == at) c[j] = 0u;
          const int id = __shfl_sync(kFullMask, lane * VPL + at, src);
          if (lane == i) my_id = id;
        }
      }
      // weights of the chosen: their logits once more, from the cache
      const float my_v = my_id >= 0 ? load_logit(static_cast<const T*>(p.logits) + t * p.ld + my_id) : -CUDART_INF_F;
      float top_v = __shfl_sync(kFullMask, my_v, 0);
      float s;
      score_row<1>(score_kind(top_v, p.sigmoid), &my_v, top_v, &s, nullptr);
      if (my_id < 0) s = 0.0f;
      const float s_all = sum_first(s, k);
      my_w = my_id >= 0 ? share_of(s, s_all) : 0.0f;
      if (my_id >= 0) atomicAdd(&s_count[my_id], 1);
    }
    if (lane < k) {
      const long long o = static_cast<long long>(t) * k + lane;
      if (p.ids32) static_cast<int*>(p.idx)[o] = my_id; else static_cast<long long*>(p.idx)[o] = my_id;
      p.weights[o] = my_w;
    }
  }
  // the block's sums, in the order of its warps
#pragma unroll
  for (int j = 0; j < VPL; ++j) sm[warp * 32 * VPL + lane * VPL + j] = acc[j];
  if (lane == 0 && live) atomicAdd(&s_live, live);
  if (bad) s_bad = 1;
  __syncthreads();
  const int busy = min(kWarps, p.T - static_cast<int>(blockIdx.x) * kWarps);  // warps that had a token
  auto block_sum = [&](int e) {
    float sum = 0.0f;
    for (int w = 0; w < busy; ++w) sum += sm[w * 32 * VPL + e];
    return sum;
  };
  unsigned long long* sums = work_sums(p.work);
  int* counts = work_counts(p.work, E);
  const bool alone = gridDim.x == 1;  // the block's sums are everybody's
  if (!alone) {
    for (int e = tid; e < E; e += blockDim.x) {
      const float sum = block_sum(e);
      if (sum > 0.0f) atomicAdd(&sums[e], __float2ull_rn(sum * p.fixed));
      if (s_count[e]) atomicAdd(&counts[e], s_count[e]);
    }
    if (tid == 0) {
      if (s_live) atomicAdd(&p.work[2], static_cast<unsigned>(s_live));
      if (s_bad) atomicOr(&p.work[1], 1u);
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(&p.work[0], 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
  }
  // every block's sums are in: results, and the work space back to zero
  const int tokens = alone ? s_live : static_cast<int>(__ldcg(&p.work[2]));
  const bool any_bad = alone ? s_bad != 0 : __ldcg(&p.work[1]) != 0u;
  float part = 0.0f;
  for (int e = tid; e < E; e += blockDim.x) {
    const int n = alone ? s_count[e] : __ldcg(&counts[e]);
    const float sum = alone ? block_sum(e) : __ull2float_rn(__ldcg(&sums[e])) * (1.0f / p.fixed);
    const float pe = any_bad ? CUDART_NAN_F : tokens ? sum / tokens : 0.0f;
    p.count[e] = n;
    p.prob[e] = pe;
    part = fmaf(static_cast<float>(n), pe, part);
    if (!alone) {
      sums[e] = 0ull;
      counts[e] = 0;
    }
  }
  part = warp_sum(part);
  if (lane == 0) s_part[warp] = part;
  __syncthreads();
  if (tid == 0) {
    float sum = 0.0f;
    for (int w = 0; w < kWarps; ++w) sum += s_part[w];
    p.count[E] = tokens;
    *p.loss = tokens ? p.coef * E / (static_cast<float>(k) * tokens) * sum : 0.0f;
    if (!alone) p.work[0] = p.work[1] = p.work[2] = 0u;
  }
}

// The lane's VPL gradients of a row, rounded to the logits' type.
template <typename T, int VPL>
__device__ __forceinline__ void store_row(T* row, int E, int lane, bool vec, const float* d) {
  constexpr int kChunk = 16 / sizeof(T);
  const int e0 = lane * VPL;
  if constexpr (VPL % kChunk == 0) {
    if (vec) {
#pragma unroll
      for (int j = 0; j < VPL; j += kChunk) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = sizeof(T) == 4 ? __float_as_uint(d[j + i]) : pack_bf16x2(d[j + (2 * i) % kChunk], d[j + (2 * i + 1) % kChunk]);
        if (e0 + j < E) *reinterpret_cast<uint4*>(row + e0 + j) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (e0 + j < E) row[e0 + j] = static_cast<T>(d[j]);
}

template <typename T, int VPL>
__global__ void __launch_bounds__(gate_warps(VPL) * 32) k_gate_backward(const GateArgs p) {
  constexpr int kWarps = gate_warps(VPL);
  extern __shared__ float sm[];  // [warps][E]: gradients of the chosen, 0 between tokens
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = p.E, k = p.k;
  float* chosen = sm + warp * 32 * VPL;
  after_previous();
  const int tokens = p.count[E];
  // sum_e p_e = 1, so c_e may be counted from any common value; from the mean
  // the difference c_e - sum p c loses fewer digits
  const float mean = static_cast<float>(k) * tokens / E;
  float c[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane * VPL + j;
    c[j] = e < E ? p.count[e] - mean : 0.0f;
    chosen[e] = 0.0f;
  }
  const bool balance = p.grad_loss && tokens;
  const float coef = balance ? *p.grad_loss * p.coef * E / (static_cast<float>(k) * tokens * tokens) : 0.0f;
  __syncwarp();
  for (int t = blockIdx.x * kWarps + warp; t < p.T; t += gridDim.x * kWarps) {
    float d[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) d[j] = 0.0f;
    if (!p.mask || p.mask[t]) {
      const T* row = static_cast<const T*>(p.logits) + t * p.ld;
      float v[VPL];
      if (balance) load_row<T, VPL>(row, E, lane, p.vec, v);
      int id = -1;
      if (p.grad_weights) {
        float dw = 0.0f, x = -CUDART_INF_F;
        if (lane < k) {
          const long long o = static_cast<long long>(t) * k + lane;
          const long long wide = load_topk_id(p.idx, o, p.ids32);
          dw = p.grad_weights[o];
          id = wide >= 0 && wide < E ? static_cast<int>(wide) : -1;
          if (id >= 0) x = load_logit(row + id);
        }
        float m = max_first(x, k), s, slope;
        score_row<1>(score_kind(m, p.sigmoid), &x, m, &s, &slope);
        if (id < 0) s = 0.0f;
        const float all = sum_first(s, k);
        const float w = id >= 0 ? share_of(s, all) : 0.0f;
        const float mean_dw = sum_first(id >= 0 ? w * dw : 0.0f, k);
        if (id >= 0) atomicAdd(chosen + id, w * slope * (dw - mean_dw));
      }
      if (balance) {
        float m = v[0];
#pragma unroll
        for (int j = 1; j < VPL; ++j) m = fmaxf(m, v[j]);
        m = warp_max(m);
        float sum = 0.0f, dot = 0.0f;
        score_row<VPL>(score_kind(m, p.sigmoid), v, m, d, v);  // 0 past E, where v is -inf; v: the slopes
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          sum += d[j];
          dot = fmaf(d[j], c[j], dot);
        }
        sum = warp_sum(sum);
        dot = warp_sum(dot);
        const float inv = sum > 0.0f ? __fdividef(1.0f, sum) : (sum == 0.0f ? 0.0f : CUDART_NAN_F);
        dot *= inv;
        const float scale = coef * inv;
#pragma unroll
        for (int j = 0; j < VPL; ++j) d[j] = scale * d[j] * v[j] * (c[j] - dot);
      }
      if (p.grad_weights) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < VPL; ++j) d[j] += chosen[lane * VPL + j];
        __syncwarp();
        if (id >= 0) chosen[id] = 0.0f;
        __syncwarp();
      }
    }
    store_row<T, VPL>(static_cast<T*>(p.grad_logits) + t * p.grad_ld, E, lane, p.grad_vec, d);
  }
}

namespace {

template <typename T, int VPL>
cudaError_t launch_vpl(const GateArgs& p, bool backward, int sms, cudaStream_t s) {
  constexpr int kWarps = gate_warps(VPL);
  const int need = (p.T + kWarps - 1) / kWarps, most = sms * ((backward ? 48 : 32) / kWarps);
  const dim3 grid(need < 1 ? 1 : need < most ? need : most), block(kWarps * 32);
  const size_t smem =
      sizeof(float) * (kWarps * 32 * VPL + (backward ? 0 : p.E + (p.groups > 1 ? kWarps * p.groups : 0)));
  return backward ? launch_early(k_gate_backward<T, VPL>, 1, grid, block, smem, s, p)
                  : launch_early(k_gate_forward<T, VPL>, 1, grid, block, smem, s, p);
}

template <typename T>
cudaError_t launch_type(const GateArgs& p, bool backward, int sms, cudaStream_t s) {
  if (p.E <= 32) return launch_vpl<T, 1>(p, backward, sms, s);
  if (p.E <= 64) return launch_vpl<T, 2>(p, backward, sms, s);
  if (p.E <= 128) return launch_vpl<T, 4>(p, backward, sms, s);
  if (p.E <= 256) return launch_vpl<T, 8>(p, backward, sms, s);
  if (p.E <= 512) return launch_vpl<T, 16>(p, backward, sms, s);
  if (p.E <= 1024) return launch_vpl<T, 32>(p, backward, sms, s);
  return launch_vpl<T, 128>(p, backward, sms, s);
}

}  // namespace

size_t gate_work_bytes(int E) { return sizeof(unsigned) * (4 + 3 * static_cast<size_t>(E)); }

cudaError_t launch_gate(const GateArgs& p, bool bf16, bool backward, int sms, cudaStream_t stream) {
  return bf16 ? launch_type<__nv_bfloat16>(p, backward, sms, stream) : launch_type<float>(p, backward, sms, stream);
}

}  // namespace ep
