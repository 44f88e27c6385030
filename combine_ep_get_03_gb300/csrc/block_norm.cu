// The norms around a block of a model, its gate and its residual scale in one pass:
//   h = residual + scale * gate . (norm(y) . post),  x = norm(h) . pre
// with norm(v) = v / sqrt(mean(v^2) + eps), and the gradients of all of it.
// Everything between loads and stores is fp32; the second norm takes h before it
// is rounded.
//
// Forward.  HBM-bound: each row of y and of the residual is read once, h and x are
// written once.  A team of 1, 2, 4, .. 16 warps takes a row, so that a thread
// holds up to 32 channels in registers across the two sums of squares; a sum
// ends in one exchange through shared memory, in a fixed order.
//
// Backward.  With hn = h rstd2, yn = y rstd1, a = grad_x pre, q = scale gate post:
//   gh = grad_h + rstd2 (a - hn m1),        m1 = mean(a hn)
//   grad_residual = gh,  grad_gate = scale gh yn post,  grad_post = scale gate gh yn,
//   grad_pre = grad_x hn,  grad_y = rstd1 (q gh - yn m2),  m2 = mean(q gh yn)
// m2 does not wait for m1: sum(q yn gh) = sum(q yn (grad_h + rstd2 a)) - m1 sum(q yn rstd2 hn),
// so one exchange per row gives both.  A block's threads own channels over all of
// its rows, so the weights' gradients are sums of the block's own; the blocks'
// partial sums are added by a second kernel in a fixed order.
#include "block_norm.cuh"
#include "experts.cuh"

namespace ep {

namespace {

__device__ __forceinline__ void unpack8(const uint4& q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(w[j]), v[2 * j + 1] = bf16_hi(w[j]);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
// Eight channels from word c of a vector or row, in fp32 or bf16.
__device__ __forceinline__ void load8(const void* p, bool fp32, long long c, float* v) {
  if (fp32) {
    const float4* f = static_cast<const float4*>(p) + 2 * c;
    const float4 a = f[0], b = f[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    unpack8(static_cast<const uint4*>(p)[c], v);
  }
}
__device__ __forceinline__ void store8(void* p, bool fp32, long long c, const float* v) {
  if (fp32) {
    float4* f = static_cast<float4*>(p) + 2 * c;
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    static_cast<uint4*>(p)[c] = pack8(v);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
  return v;
}

__device__ __forceinline__ void team_barrier(int team, int threads) {
  asm volatile("bar.sync %0, %1;" : : "r"(team + 1), "r"(threads) : "memory");
}

// Sum over a team of `warps` warps; `part` holds a word for each.
__device__ __forceinline__ float team_sum(float v, float* part, int team, int warps) {
  v = warp_sum(v);
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % warps;
  if (lane == 0) part[warp] = v;
  team_barrier(team, warps * 32);
  float s = 0.0f;
  for (int w = 0; w < warps; ++w) s += part[w];
  return s;
}

}  // namespace

// kWords: 16-byte words of bf16 that a thread holds of each row.
template <int kWords, bool kRes32>
__global__ void k_block_norm(const BlockNormArgs a, int warps) {
  __shared__ float part[2][32];
  after_previous();
  const int per_team = warps * 32, teams = blockDim.x / per_team;
  const int team = threadIdx.x / per_team, tid = threadIdx.x % per_team;
  float* sums[2] = {part[0] + team * warps, part[1] + team * warps};
  const int words = a.H >> 3;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  for (long long t = static_cast<long long>(blockIdx.x) * teams + team; t < a.T;
       t += static_cast<long long>(gridDim.x) * teams) {
    const long long row = t * words;
    if (a.mask && !a.mask[t]) {
      const float zero[8] = {};
      for (int c = tid; c < words; c += per_team) {
        if (a.y) store8(a.new_residual, kRes32, row + c, zero);
        if (a.x) store8(a.x, false, row + c, zero);
      }
      if (tid == 0 && a.rstd) {
        if (a.post) a.rstd[t] = 0.0f;
        if (a.x) a.rstd[a.T + t] = 0.0f;
      }
      continue;
    }
    uint4 y[kWords];
    float h[kWords][8];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int c = tid + i * per_team;
      y[i] = make_uint4(0, 0, 0, 0);
      if (c < words && a.y) y[i] = ld_stream(static_cast<const uint16_t*>(a.y) + 8 * (row + c));
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int c = tid + i * per_team;
      if (c < words) {
        load8(a.residual, kRes32, row + c, h[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
      }
    }
    if (a.y) {
      float r1 = 1.0f;
      if (a.post) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          float v[8];
          unpack8(y[i], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
        }
        r1 = rsqrtf(fmaf(team_sum(s, sums[0], team, warps), inv_h, a.eps));
        if (tid == 0 && a.rstd) a.rstd[t] = r1;
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int c = tid + i * per_team;
        if (c < words) {
          float v[8], w[8];
          unpack8(y[i], v);
          if (a.post) {
            load8(a.post, a.weight32, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= r1 * w[j];
          }
          if (a.gate) {
            load8(a.gate, a.weight32 && !a.gate_per_token, a.gate_per_token ? row + c : c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= w[j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] = fmaf(a.scale, v[j], h[i][j]);
          store8(a.new_residual, kRes32, row + c, h[i]);
        }
      }
    }
    if (a.x) {
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(h[i][j], h[i][j], s);
      const float r2 = rsqrtf(fmaf(team_sum(s, sums[1], team, warps), inv_h, a.eps));
      if (tid == 0 && a.rstd) a.rstd[a.T + t] = r2;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int c = tid + i * per_team;
        if (c < words) {
          float w[8];
          load8(a.pre, a.weight32, c, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] *= h[i][j] * r2;
          store8(a.x, false, row + c, w);
        }
      }
    }
  }
}

namespace {

constexpr int kBackThreads = 512, kBackWarps = kBackThreads / 32;

}  // namespace

// Partial sums of the weights' gradients in shared memory, [3][H] (pre, post,
// gate), a thread's channels its own.
template <bool kRes32>
__global__ void __launch_bounds__(kBackThreads, 1) k_block_norm_backward(const BlockNormBackwardArgs a) {
  extern __shared__ float4 own4[];
  float* own = reinterpret_cast<float*>(own4);
  __shared__ float part[2][3][kBackWarps];
  after_previous();
  const BlockNormArgs& n = a.n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = n.H >> 3;
  const float inv_h = 1.0f / static_cast<float>(n.H);
  const bool pre = a.grad_x != nullptr, block = a.grad_y || a.grad_gate || a.grad_post;
  const bool post = block && n.post, vector = a.grad_gate && !n.gate_per_token;
  for (int c = tid; c < words; c += kBackThreads)
    for (int k = 0; k < 3; ++k)
      for (int j = 0; j < 8; ++j) own[k * n.H + 8 * c + j] = 0.0f;
  int turn = 0;
  for (long long t = blockIdx.x; t < n.T; t += gridDim.x) {
    const long long row = t * words;
    if (n.mask && !n.mask[t]) {
      const float zero[8] = {};
      for (int c = tid; c < words; c += kBackThreads) {
        if (a.grad_residual) store8(a.grad_residual, kRes32, row + c, zero);
        if (a.grad_y) store8(a.grad_y, false, row + c, zero);
        if (a.grad_gate && n.gate_per_token) store8(a.grad_gate, false, row + c, zero);
      }
      continue;
    }
    const float r1 = post ? n.rstd[t] : 1.0f, r2 = pre ? n.rstd[n.T + t] : 0.0f;
    float m1 = 0.0f, m2 = 0.0f;
    if (pre || (post && a.grad_y)) {
      float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
      for (int c = tid; c < words; c += kBackThreads) {
        float g[8] = {}, hn[8] = {};
        if (a.grad_new) load8(a.grad_new, kRes32, row + c, g);
        if (pre) {
          float x[8], w[8];
          load8(n.new_residual, kRes32, row + c, hn);
          load8(a.grad_x, false, row + c, x);
          load8(n.pre, n.weight32, c, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            hn[j] *= r2;
            x[j] *= w[j];
            s1 = fmaf(x[j], hn[j], s1);
            g[j] = fmaf(r2, x[j], g[j]);
          }
        }
        if (post) {
          float y[8], w[8], q[8];
          load8(n.y, false, row + c, y);
          load8(n.post, n.weight32, c, w);
          if (n.gate) load8(n.gate, n.weight32 && !n.gate_per_token, n.gate_per_token ? row + c : c, q);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float u = (n.gate ? q[j] : 1.0f) * w[j] * (y[j] * r1);
            s2 = fmaf(u, g[j], s2);
            s3 = fmaf(u, hn[j], s3);
          }
        }
      }
      s1 = warp_sum(s1), s2 = warp_sum(s2), s3 = warp_sum(s3);
      if (lane == 0) part[turn][0][warp] = s1, part[turn][1][warp] = s2, part[turn][2][warp] = s3;
      __syncthreads();
      s1 = s2 = s3 = 0.0f;
#pragma unroll
      for (int w = 0; w < kBackWarps; ++w) s1 += part[turn][0][w], s2 += part[turn][1][w], s3 += part[turn][2][w];
      turn ^= 1;
      m1 = s1 * inv_h;
      m2 = n.scale * inv_h * fmaf(-m1 * r2, s3, s2);
    }
    for (int c = tid; c < words; c += kBackThreads) {
      float g[8] = {};
      if (a.grad_new) load8(a.grad_new, kRes32, row + c, g);
      if (pre) {
        float x[8], w[8], hn[8];
        load8(n.new_residual, kRes32, row + c, hn);
        load8(a.grad_x, false, row + c, x);
        load8(n.pre, n.weight32, c, w);
        float* o = own + 8 * c;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          hn[j] *= r2;
          if (a.grad_pre) o[j] = fmaf(x[j], hn[j], o[j]);
          g[j] = fmaf(r2, fmaf(-hn[j], m1, x[j] * w[j]), g[j]);
        }
      }
      if (a.grad_residual) store8(a.grad_residual, kRes32, row + c, g);
      if (!block) continue;
      float y[8] = {}, w[8], q[8];
      if (post || a.grad_gate) load8(n.y, false, row + c, y);
      if (post) load8(n.post, n.weight32, c, w);
      if (n.gate) load8(n.gate, n.weight32 && !n.gate_per_token, n.gate_per_token ? row + c : c, q);
      float dg[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float yn = y[j] * r1, gn = n.scale * g[j];
        dg[j] = gn * (post ? yn * w[j] : yn);
        const float u = n.gate ? gn * q[j] : gn;
        if (post && a.grad_post) own[n.H + 8 * c + j] = fmaf(u, yn, own[n.H + 8 * c + j]);
        if (vector) own[2 * n.H + 8 * c + j] += dg[j];
        g[j] = post ? r1 * fmaf(-yn, m2, u * w[j]) : u;
      }
      if (a.grad_gate && n.gate_per_token) store8(a.grad_gate, false, row + c, dg);
      if (a.grad_y) store8(a.grad_y, false, row + c, g);
    }
  }
  for (int c = tid; c < words; c += kBackThreads)
    for (int k = 0; k < 3; ++k)
      if (k == 0 ? a.grad_pre != nullptr : k == 1 ? a.grad_post != nullptr : vector)
        for (int j = 0; j < 8; ++j)
          a.partial[(static_cast<long long>(blockIdx.x) * 3 + k) * n.H + 8 * c + j] = own[k * n.H + 8 * c + j];
}

// out[k][i] = sum over blocks of partial[block][k][i], eight runs of blocks side by side.
__global__ void __launch_bounds__(256) k_block_norm_sums(const float* partial, int blocks, int H, float* pre, float* post,
                                                         float* gate) {
  __shared__ float4 runs[8][32];
  after_previous();
  float* out = blockIdx.y == 0 ? pre : blockIdx.y == 1 ? post : gate;
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int i = (blockIdx.x * 32 + lane) * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (out && i < H) {
#pragma unroll 4
    for (int b = run; b < blocks; b += 8) {
      const float4 v = *reinterpret_cast<const float4*>(partial + (static_cast<long long>(b) * 3 + blockIdx.y) * H + i);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
  }
  runs[run][lane] = s;
  __syncthreads();
  if (run == 0 && out && i < H) {
    for (int r = 1; r < 8; ++r) {
      const float4 v = runs[r][lane];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    *reinterpret_cast<float4*>(out + i) = s;
  }
}

cudaError_t launch_block_norm(const BlockNormArgs& a, bool res32, int sms, cudaStream_t stream) {
  const int words = a.H / 8;
  int warps = 1;
  while (warps * 32 * 4 < words) warps *= 2;
  const int per_thread = (words + warps * 32 - 1) / (warps * 32);
  const int threads = warps < 8 ? 256 : warps * 32, teams = threads / (warps * 32);
  using Kernel = void (*)(BlockNormArgs, int);
  static const Kernel kernels[2][4] = {
      {k_block_norm<1, false>, k_block_norm<2, false>, k_block_norm<3, false>, k_block_norm<4, false>},
      {k_block_norm<1, true>, k_block_norm<2, true>, k_block_norm<3, true>, k_block_norm<4, true>}};
  const long long need = (static_cast<long long>(a.T) + teams - 1) / teams, most = static_cast<long long>(sms) * (threads == 256 ? 3 : 1);
  return launch_early(kernels[res32][per_thread - 1], 1, dim3(static_cast<unsigned>(need < most ? need : most)),
                      dim3(threads), 0, stream, a, warps);
}

cudaError_t launch_block_norm_backward(const BlockNormBackwardArgs& a, bool res32, int sms, cudaStream_t stream) {
  auto kernel = res32 ? k_block_norm_backward<true> : k_block_norm_backward<false>;
  static std::atomic<unsigned long long> ready[2];  // devices set up, a bit each
  cudaError_t e = set_up_kernel(reinterpret_cast<const void*>(kernel), ready[res32], 0);
  if (e != cudaSuccess) return e;
  int blocks = sms < kBlockNormMaxBlocks ? sms : kBlockNormMaxBlocks;
  if (blocks > a.n.T) blocks = a.n.T;
  e = launch_early(kernel, 1, dim3(blocks), dim3(kBackThreads), sizeof(float) * 3 * a.n.H, stream, a);
  const bool vector = a.grad_gate && !a.n.gate_per_token;
  if (e != cudaSuccess || !(a.grad_pre || a.grad_post || vector)) return e;
  return launch_early(k_block_norm_sums, 1, dim3((a.n.H + 127) / 128, 3), dim3(256), 0, stream,
                      static_cast<const float*>(a.partial), blocks, a.n.H, a.grad_pre, a.grad_post,
                      vector ? static_cast<float*>(a.grad_gate) : nullptr);
}

}  // namespace ep
