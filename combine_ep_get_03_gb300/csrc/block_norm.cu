// The norms around a block of a model, its gate and its residual scale in one pass:
//   h = residual + scale * gate . (norm(y) . post),  x = norm(h) . pre
// with norm(v) = v / sqrt(mean(v^2) + eps), and the gradients of all of it.
// Everything between loads and stores is fp32; the second norm takes h before it
// is rounded.
//
// Both are HBM-bound: each tensor's row is read once and each result's written once.
// A team of warps takes a row, two 8-channel words a thread (one in most of the
// backward's rows up to 4096); short rows leave room
// for several teams in a block, one block an SM.  A sum over a row ends in an exchange through
// shared memory, in a fixed order.
//
// Forward: two sums a row, of y^2 and of h^2.  16 384 tokens of 7168 channels: fp32
// residual 221 us (6.4 TB/s), bf16 146; 4 096 channels fp32 124; one token 3.7 us in
// a graph.  Rows in registers beyond 8192 channels: 4 096 tokens of 12 288 bf16 85 us, fp32
// 104; of 16 384 90 and 141 (5.7 TB/s).  (Up to 8192, rows loaded to registers, a block of
// 8 warps a row: 226 us with the next rows fetched to L2, 158, 132 and 4.9; 240, 191
// without.  The second sum exchanged with the next row's first, one barrier a row: 245,
// 150, 145 and 3.9.)
//
// Backward.  8 192 tokens of 7168, gate a vector: bf16 115 us (6.1 TB/s), fp32 165; 4 099
// of 2048, fp32, gate per token: 39 us, some 8 of them two launches' start and end.  Beyond
// 8192 channels rows are read twice: 4 096 of 12 288 bf16 270 us, fp32 277; of 16 384 369
// and 415.
// With hn = h rstd2, yn = y rstd1, a = grad_x pre, q = scale gate post:
//   gh = grad_h + rstd2 (a - hn m1),        m1 = mean(a hn)
//   grad_residual = gh,  grad_gate = scale gh yn post,  grad_post = scale gate gh yn,
//   grad_pre = grad_x hn,  grad_y = rstd1 (q gh - yn m2),  m2 = mean(q gh yn)
// m2 does not wait for m1: sum(q yn gh) = sum(q yn (grad_h + rstd2 a)) - m1 sum(q yn rstd2 hn),
// so one exchange per row gives both.  A block's threads own channels over all of
// its rows, so the weights' gradients are sums of the block's own; the blocks'
// partial sums are added by a second kernel in a fixed order.
#include "block_norm.cuh"
#include "experts.cuh"
#include "pairs.cuh"

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

__device__ __forceinline__ void load8(const void* p, bool fp32, long long c, float2* v) {
  if (fp32) {
    const float4* f = static_cast<const float4*>(p) + 2 * c;
    const float4 a = f[0], b = f[1];
    v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
  } else {
    const uint4 q = static_cast<const uint4*>(p)[c];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float2(bf16_lo(w[j]), bf16_hi(w[j]));
  }
}
__device__ __forceinline__ void store8(void* p, bool fp32, long long c, const float2* v) {
  if (fp32) {
    float4* f = static_cast<float4*>(p) + 2 * c;
    f[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    f[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  } else {
    static_cast<uint4*>(p)[c] = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                           pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
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

constexpr int kRingThreads = 512, kRingWarps = kRingThreads / 32;
constexpr int kWordsEach = 2;                               // 8-channel words of a row that a thread owns
constexpr int kRingHidden = kRingThreads * kWordsEach * 8;  // rows beyond take the kernels for long rows
constexpr int kMaxStages = 4;
constexpr int kRingAlign = 128;  // of the dynamic shared memory, and so of what lies before it
// Warps of the backward pass's other instance of two words a thread.  A thread has 128
// registers in both, but what the compiler makes of them differs (8192 rows, us, 14
// against 16 warps at most: bf16 7168 115 and 143, 5120 97 and 122; fp32 7168 165 and 178, 5120 132
// and 122; bf16 with a gate per token 7168 188 and 197, 5120 159 and 161; fp32 with one, which
// therefore takes 16, 247 and 201, 192 and 166).
constexpr int kNarrowWarps = 14;

// What a thread takes for a row whose copies it waited for in vain.  It asks for no
// more copies then, so that no barrier's rounds mix, and waits in vain for later rows too.
__device__ __forceinline__ float2 lost() { return both(__int_as_float(0x7fc00000)); }

// Barriers and partial sums of a block's teams.
struct RingShared {
  uint64_t full[kRingWarps][kMaxStages];
  float4 part[kRingWarps][2][kRingWarps];  // [team][parity][warp of the team], zeros past the team
  int quit;
};

}  // namespace

// Forward: a team of warps takes a row at a time; its tensors' rows arrive by bulk
// copies in a ring of stages in shared memory, and a thread keeps its channels'
// weights in registers over all rows.  The first barrier of a row's sums says that
// the stage of the row before has been read, so its refill needs no other.
// kY: there is a block behind; kToken: its gate comes per token; kMask: there may be
// padding tokens.  (One kernel with and without: 16 384 x 7168 fp32 without 221 -> 227 us,
// but with a gate per token 272 -> 263, so that is always the one with.)
template <bool kRes32, bool kY, bool kToken, bool kMask>
__global__ void __launch_bounds__(kRingThreads, 1) k_block_norm(const BlockNormArgs a, int warps, int num_stages) {
  extern __shared__ __align__(kRingAlign) unsigned char ring[];
  __shared__ RingShared s;
  const int lane = threadIdx.x & 31, teams = blockDim.x / (warps * 32);
  const int team = threadIdx.x / (warps * 32), threads = warps * 32, tid = threadIdx.x % threads, warp = tid >> 5;
  const int words = a.H >> 3;
  constexpr int kR = kRes32 ? 4 : 2, kCopies = 1 + kY + kToken;
  const int o_y = kR * a.H, o_g = o_y + (kY ? 2 * a.H : 0), stage_bytes = o_g + (kToken ? 2 * a.H : 0);
  unsigned char* stages = ring + static_cast<size_t>(team) * num_stages * stage_bytes;
  uint64_t* full = s.full[team];
  // the i-th tensor's rows are copied by lane 0 of warp i % warps
  unsigned mine = 0;
  for (int i = 0; lane == 0 && i < kCopies; ++i)
    if (i % warps == warp) mine |= 1u << i;
  if (tid == 0) {
    for (int i = 0; i < num_stages; ++i) mbar_init(&full[i], kCopies);
    s.quit = 0;
    mbar_init_fence();
  }
  if (tid < 32) s.part[team][tid >> 4][tid & 15] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  after_previous();
  __syncthreads();
  const long long step = static_cast<long long>(gridDim.x) * teams;
  const long long first = static_cast<long long>(blockIdx.x) * teams + team;
  auto fetch = [&](long long t, int st) {
    if (t >= a.T || !mine) return;
    unsigned char* d = stages + static_cast<size_t>(st) * stage_bytes;
    const long long at = t * a.H;
    int i = 0;
    auto copy = [&](int to, const void* from, int size) {
      if (!(mine >> i++ & 1)) return;
      mbar_arrive_expect_tx(&full[st], size * a.H);
      bulk_load(d + to, static_cast<const char*>(from) + at * size, size * a.H, &full[st]);
    };
    copy(0, a.residual, kR);
    if (kY) copy(o_y, a.y, 2);
    if (kToken) copy(o_g, a.gate, 2);
  };
  for (int i = 0; i < num_stages; ++i) fetch(first + i * step, i);

  // the channels' constants: pre, and q = scale post (times gate where it is a vector)
  const bool post = kY && a.post, pre = a.x != nullptr;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  float2 wp[kWordsEach][4], q[kWordsEach][4];
#pragma unroll
  for (int k = 0; k < kWordsEach; ++k) {
    const int c = tid + k * threads;
#pragma unroll
    for (int j = 0; j < 4; ++j) wp[k][j] = both(0.0f), q[k][j] = both(a.scale);
    if (c >= words) continue;
    float2 v[4];
    if (pre) load8(a.pre, a.weight32, c, wp[k]);
    if (post) {
      load8(a.post, a.weight32, c, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[k][j] = mul2(q[k][j], v[j]);
    }
    if (kY && !kToken && a.gate) {
      load8(a.gate, a.weight32, c, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[k][j] = mul2(q[k][j], v[j]);
    }
  }

  int st = 0, phase = 0, turn = 0;
  // sum over the team; the other of the two sets of parts at each call
  auto sum = [&](float2 v) {
    float f = warp_sum(v.x + v.y);
    if (warps == 1) return f;
    float4* part = s.part[team][turn];
    turn ^= 1;
    if (lane == 0) part[warp].x = f;
    team_barrier(team, threads);
    f = part[lane & 15].x;
#pragma unroll
    for (int b = 8; b; b >>= 1) f += __shfl_xor_sync(kFullMask, f, b);
    return f;
  };
  bool next_live = !kMask || !a.mask || first >= a.T || a.mask[first];
  for (long long t = first; t < a.T; t += step) {
    const bool live = next_live;
    if (kMask && a.mask && t + step < a.T) next_live = a.mask[t + step];
    const unsigned char* d = stages + static_cast<size_t>(st) * stage_bytes;
    const bool landed = wait_or_quit(&full[st], phase, &s.quit, nullptr);
    auto refill = [&]() {
      if (t != first) fetch(t + (num_stages - 1) * step, st ? st - 1 : num_stages - 1);
    };
    const long long row = t * words;
    if (kMask && !live) {  // zeros, whatever the weights are
      if (warps > 1) team_barrier(team, threads);
      else __syncwarp();
      if (!landed) mine = 0;
      refill();
      const float zero[8] = {};
      for (int c = tid; c < words; c += threads) {
        if (kY) store8(a.new_residual, kRes32, row + c, zero);
        if (pre) store8(a.x, false, row + c, zero);
      }
      if (tid == 0 && a.rstd) {
        if (post) a.rstd[t] = 0.0f;
        if (pre) a.rstd[a.T + t] = 0.0f;
      }
      __syncwarp();
      if (++st == num_stages) st = 0, phase ^= 1;
      continue;
    }
    float2 h[kWordsEach][4], y[kY ? kWordsEach : 1][4];
    float2 t1 = both(0.0f);
#pragma unroll
    for (int k = 0; k < kWordsEach; ++k) {
      const int c = tid + k * threads;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[k][j] = both(0.0f);
        if (kY) y[k][j] = both(0.0f);
      }
      if (c >= words) continue;
      load8(d, kRes32, c, h[k]);
      if (kY) {
        load8(d + o_y, false, c, y[k]);
        if (post) {
#pragma unroll
          for (int j = 0; j < 4; ++j) t1 = fma2(y[k][j], y[k][j], t1);
        }
      }
    }
    if (!landed) {  // a copy that never came: NaN, not old values, in the sums too
      mine = 0;
      t1 = lost();
#pragma unroll
      for (int k = 0; k < kWordsEach; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k][j] = lost();
    }
    float r1 = 1.0f;
    if (post) r1 = rsqrtf(fmaf(sum(t1), inv_h, a.eps));
    if (post) refill();
    if (kY) {
      if (post && tid == 0 && a.rstd) a.rstd[t] = r1;
#pragma unroll
      for (int k = 0; k < kWordsEach; ++k) {
        const int c = tid + k * threads;
        if (c >= words) continue;
        float2 u[4];
        if (kToken) load8(d + o_g, false, c, u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 v = mul2(y[k][j], both(r1));
          if (kToken) v = mul2(v, u[j]);
          h[k][j] = fma2(q[k][j], v, h[k][j]);
        }
        store8(a.new_residual, kRes32, row + c, h[k]);
      }
    }
    if (pre) {
      float2 t2 = both(0.0f);
#pragma unroll
      for (int k = 0; k < kWordsEach; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) t2 = fma2(h[k][j], h[k][j], t2);
      const float r2 = rsqrtf(fmaf(sum(t2), inv_h, a.eps));
      if (!post) refill();
      if (tid == 0 && a.rstd) a.rstd[a.T + t] = r2;
#pragma unroll
      for (int k = 0; k < kWordsEach; ++k) {
        const int c = tid + k * threads;
        if (c >= words) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k][j] = mul2(mul2(h[k][j], both(r2)), wp[k][j]);
        store8(a.x, false, row + c, h[k]);
      }
    } else if (!post) {
      if (warps > 1) team_barrier(team, threads);
      else __syncwarp();
      refill();
    }
    __syncwarp();
    if (++st == num_stages) st = 0, phase ^= 1;
  }
}

// The forward pass of rows too long for that: a block a row, the row in its threads'
// registers.  kWords: 16-byte words of bf16 that a thread holds of each row.
template <int kWords, bool kRes32>
__global__ void __launch_bounds__(kRingThreads) k_block_norm_long(const BlockNormArgs a) {
  __shared__ float part[2][kRingWarps];
  after_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = a.H >> 3;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  int turn = 0;
  auto sum = [&](float v) {  // in the other of the two sets of parts at each call
    float* parts = part[turn];
    turn ^= 1;
    v = warp_sum(v);
    if (lane == 0) parts[warp] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kRingWarps; ++w) v += parts[w];
    return v;
  };
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const long long row = t * words;
    if (a.mask && !a.mask[t]) {
      const float zero[8] = {};
      for (int c = tid; c < words; c += kRingThreads) {
        if (a.y) store8(a.new_residual, kRes32, row + c, zero);
        if (a.x) store8(a.x, false, row + c, zero);
      }
      if (tid == 0 && a.rstd) {
        if (a.post) a.rstd[t] = 0.0f;
        if (a.x) a.rstd[a.T + t] = 0.0f;
      }
      continue;
    }
    if (tid == 0 && t + gridDim.x < a.T) {
      // the block's next rows on their way to L2
      const long long next = (t + gridDim.x) * a.H;
      constexpr int kR = kRes32 ? 4 : 2;
      prefetch_l2_bulk(static_cast<const char*>(a.residual) + next * kR, a.H * kR);
      if (a.y) prefetch_l2_bulk(static_cast<const uint16_t*>(a.y) + next, a.H * 2);
      if (a.gate_per_token) prefetch_l2_bulk(static_cast<const uint16_t*>(a.gate) + next, a.H * 2);
    }
    uint4 y[kWords];
    float h[kWords][8];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int c = tid + i * kRingThreads;
      y[i] = make_uint4(0, 0, 0, 0);
      if (c < words && a.y) y[i] = ld_stream(static_cast<const uint16_t*>(a.y) + 8 * (row + c));
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int c = tid + i * kRingThreads;
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
        r1 = rsqrtf(fmaf(sum(s), inv_h, a.eps));
        if (tid == 0 && a.rstd) a.rstd[t] = r1;
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int c = tid + i * kRingThreads;
        if (c >= words) continue;
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
    if (!a.x) continue;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(h[i][j], h[i][j], s);
    const float r2 = rsqrtf(fmaf(sum(s), inv_h, a.eps));
    if (tid == 0 && a.rstd) a.rstd[a.T + t] = r2;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int c = tid + i * kRingThreads;
      if (c >= words) continue;
      float w[8];
      load8(a.pre, a.weight32, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= h[i][j] * r2;
      store8(a.x, false, row + c, w);
    }
  }
}

// Backward: the same teams and rings, of two stages or more, each row read twice: for
// the sums, and for the results.  The barrier of a row's sums says that the stage of
// the row before has been read, so its refill needs no other; with an fp32 residual, where a long
// row leaves room for two stages only, a second barrier lets the refill start half a
// row earlier (8192 x 7168: 228 -> 166 us; with a bf16 residual, three stages, 116 ->
// 146).  Each tensor's copy is asked for by a warp of its own.
// kPre: x's gradient takes part; kY: y is needed (a norm behind the block or its
// gate's gradient); kToken: the gate comes per token.
// kThreads: the most that the block has.
// kWords: the 8-channel words of a row that a thread owns.
template <int kThreads, int kWords, bool kRes32, bool kPre, bool kY, bool kToken>
__global__ void __launch_bounds__(kThreads, 1)
    k_block_norm_backward(const BlockNormBackwardArgs a, int warps, int num_stages) {
  extern __shared__ __align__(kRingAlign) unsigned char ring[];
  __shared__ RingShared s;
  const BlockNormArgs& n = a.n;
  const int lane = threadIdx.x & 31, teams = blockDim.x / (warps * 32);
  const int team = threadIdx.x / (warps * 32), threads = warps * 32, tid = threadIdx.x % threads, warp = tid >> 5;
  const int words = n.H >> 3;
  constexpr int kR = kRes32 ? 4 : 2;
  constexpr bool kEarly = kRes32;
  const bool grad_new = a.grad_new != nullptr;
  const int o_h = grad_new ? kR * n.H : 0, o_x = o_h + (kPre ? kR * n.H : 0), o_y = o_x + (kPre ? 2 * n.H : 0);
  const int o_g = o_y + (kY ? 2 * n.H : 0), stage_bytes = o_g + (kToken ? 2 * n.H : 0);
  unsigned char* stages = ring + static_cast<size_t>(team) * num_stages * stage_bytes;
  uint64_t* full = s.full[team];
  const int copies = grad_new + 2 * kPre + kY + kToken;
  // the i-th tensor's rows are copied by lane 0 of warp i % warps
  unsigned mine = 0;
  for (int i = 0; lane == 0 && i < copies; ++i)
    if (i % warps == warp) mine |= 1u << i;
  if (tid == 0) {
    // an mbarrier counts from 1; where nothing is read nobody waits
    for (int i = 0; i < num_stages; ++i) mbar_init(&full[i], copies ? copies : 1);
    s.quit = 0;
    mbar_init_fence();
  }
  if (tid < 32) s.part[team][tid >> 4][tid & 15] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  after_previous();
  __syncthreads();
  const long long step = static_cast<long long>(gridDim.x) * teams;
  const long long first = static_cast<long long>(blockIdx.x) * teams + team;
  // row t's copies into stage st
  auto fetch = [&](long long t, int st) {
    if (t >= n.T || !mine) return;
    unsigned char* d = stages + static_cast<size_t>(st) * stage_bytes;
    const long long at = t * n.H;
    int i = 0;
    auto copy = [&](int to, const void* from, int size) {
      if (!(mine >> i++ & 1)) return;
      mbar_arrive_expect_tx(&full[st], size * n.H);
      bulk_load(d + to, static_cast<const char*>(from) + at * size, size * n.H, &full[st]);
    };
    if (grad_new) copy(0, a.grad_new, kR);
    if (kPre) copy(o_h, n.new_residual, kR), copy(o_x, a.grad_x, 2);
    if (kY) copy(o_y, n.y, 2);
    if (kToken) copy(o_g, n.gate, 2);
  };
  for (int i = 0; i < num_stages; ++i) fetch(first + i * step, i);

  // the channels' constants: pre, and q = scale post (times gate where it is a vector)
  const bool post = kY && n.post;
  const float inv_h = 1.0f / static_cast<float>(n.H);
  float2 wp[kPre ? kWords : 1][4], q[kWords][4];
  float2 sum_pre[kPre ? kWords : 1][4], sum_y[kY ? kWords : 1][4];
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    const int c = tid + k * threads;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q[k][j] = both(n.scale);
      if (kPre) wp[k][j] = sum_pre[k][j] = both(0.0f);
      if (kY) sum_y[k][j] = both(0.0f);
    }
    if (c < words) {
      float2 v[4];
      if (kPre) load8(n.pre, n.weight32, c, wp[k]);
      if (n.post && kY) {
        load8(n.post, n.weight32, c, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[k][j] = mul2(q[k][j], v[j]);
      }
      if (n.gate && !n.gate_per_token) {
        load8(n.gate, n.weight32, c, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[k][j] = mul2(q[k][j], v[j]);
      }
    }
  }

  int st = 0, phase = 0, turn = 0;
  float next1 = 1.0f, next2 = 0.0f;
  bool next_live = true;
  if (first < n.T) {
    if (n.mask) next_live = n.mask[first];
    if (post) next1 = n.rstd[first];
    if (kPre) next2 = n.rstd[n.T + first];
  }
  for (long long t = first; t < n.T; t += step) {
    const float r1 = next1, r2 = next2;
    const bool live = next_live;
    if (t + step < n.T) {
      if (n.mask) next_live = n.mask[t + step];
      if (post) next1 = n.rstd[t + step];
      if (kPre) next2 = n.rstd[n.T + t + step];
    }
    const unsigned char* d = stages + static_cast<size_t>(st) * stage_bytes;
    const bool landed = !copies || wait_or_quit(&full[st], phase, &s.quit, nullptr);
    float2 g[kWords][4];
    float2 t1 = both(0.0f), t2 = t1, t3 = t1;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const int c = tid + k * threads;
#pragma unroll
      for (int j = 0; j < 4; ++j) g[k][j] = both(0.0f);
      if (c < words && live) {
        float2 hn[4], x[4], y[4], u[4];
        if (grad_new) load8(d, kRes32, c, g[k]);
        if (kPre) load8(d + o_h, kRes32, c, hn), load8(d + o_x, false, c, x);
        if (kY) load8(d + o_y, false, c, y);
        if (kY && kToken) load8(d + o_g, false, c, u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // sums of a h, u g and u h: rstd2 and rstd1 come in behind them
          if (kPre) {
            x[j] = mul2(x[j], wp[k][j]);
            t1 = fma2(x[j], hn[j], t1);
            g[k][j] = fma2(both(r2), x[j], g[k][j]);
          }
          if (kY) {
            y[j] = mul2(y[j], q[k][j]);
            if (kToken) y[j] = mul2(y[j], u[j]);
            t2 = fma2(y[j], g[k][j], t2);
            if (kPre) t3 = fma2(y[j], hn[j], t3);
          }
        }
      }
    }
    if (!landed) {  // a copy that never came: NaN, not old values, in the sums too
      mine = 0;
      t1 = t2 = lost();
#pragma unroll
      for (int k = 0; k < kWords; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g[k][j] = lost();
          if (kPre) sum_pre[k][j] = lost();
        }
    }
    float s1 = t1.x + t1.y, s2 = t2.x + t2.y, s3 = t3.x + t3.y;
    if (kPre) s1 = warp_sum(s1);
    if (kY) s2 = warp_sum(s2);
    if (kPre && kY) s3 = warp_sum(s3);
    if (warps > 1) {
      float4* part = s.part[team][turn];
      if (lane == 0) part[warp] = make_float4(s1, s2, s3, 0.0f);
      team_barrier(team, threads);
      // sixteen parts, each half of the warp the same
      const float4 p = part[lane & 15];
      s1 = p.x, s2 = p.y, s3 = p.z;
#pragma unroll
      for (int b = 8; b; b >>= 1) {
        if (kPre) s1 += __shfl_xor_sync(kFullMask, s1, b);
        if (kY) s2 += __shfl_xor_sync(kFullMask, s2, b);
        if (kPre && kY) s3 += __shfl_xor_sync(kFullMask, s3, b);
      }
      turn ^= 1;
    } else {
      __syncwarp();
    }
    // the row before has been read by everyone
    if (!kEarly && t != first) fetch(t + (num_stages - 1) * step, st ? st - 1 : num_stages - 1);
    const float m1 = s1 * r2 * inv_h * r2;
    const float m2 = post ? inv_h * r1 * fmaf(-m1 * r2, s3, s2) : 0.0f;
    const long long row = t * words;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const int c = tid + k * threads;
      if (c >= words) continue;
      if (!live) {
        const float zero[8] = {};
        if (a.grad_residual) store8(a.grad_residual, kRes32, row + c, zero);
        if (a.grad_y) store8(a.grad_y, false, row + c, zero);
        if (kToken && a.grad_gate) store8(a.grad_gate, false, row + c, zero);
        continue;
      }
      float2 u[4], y[4];
      if (kPre) {
        float2 hn[4], x[4];
        load8(d + o_h, kRes32, c, hn);
        load8(d + o_x, false, c, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          hn[j] = mul2(hn[j], both(r2));
          sum_pre[k][j] = fma2(x[j], hn[j], sum_pre[k][j]);
          g[k][j] = fma2(hn[j], both(-m1), g[k][j]);
        }
      }
      if (kY) load8(d + o_y, false, c, y);
      if (kToken) load8(d + o_g, false, c, u);
      if (a.grad_residual) store8(a.grad_residual, kRes32, row + c, g[k]);
      if (kY) {
        float2 dg[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = mul2(y[j], both(r1));
          if (kToken) {
            const float2 v = mul2(g[k][j], y[j]);
            dg[j] = mul2(q[k][j], v);
            sum_y[k][j] = fma2(u[j], v, sum_y[k][j]);
            g[k][j] = mul2(mul2(q[k][j], u[j]), g[k][j]);
          } else {
            sum_y[k][j] = fma2(g[k][j], y[j], sum_y[k][j]);
            g[k][j] = mul2(q[k][j], g[k][j]);
          }
          g[k][j] = mul2(both(r1), fma2(y[j], both(-m2), g[k][j]));
        }
        if (kToken && a.grad_gate) store8(a.grad_gate, false, row + c, dg);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g[k][j] = mul2(q[k][j], g[k][j]);
          if (kToken) g[k][j] = mul2(u[j], g[k][j]);
        }
      }
      if (a.grad_y) store8(a.grad_y, false, row + c, g[k]);
    }
    if (kEarly) {
      if (warps > 1) team_barrier(team, threads);
      else __syncwarp();
      fetch(t + num_stages * step, st);
    }
    __syncwarp();
    if (++st == num_stages) st = 0, phase ^= 1;
  }

  // the block's sums: its teams', in their order
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    const int c = tid + k * threads;
    if (c >= words) continue;
    float* to = teams == 1 ? a.partial + static_cast<long long>(blockIdx.x) * 2 * n.H : sums + team * 2 * n.H;
    if (kPre && a.grad_pre) store8(to, true, c, sum_pre[k]);
    if (kY && a.sum_y) store8(to + n.H, true, c, sum_y[k]);
  }
  if (teams == 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * n.H; i += blockDim.x) {
    if (i < n.H ? !(kPre && a.grad_pre) : !(kY && a.sum_y)) continue;
    float v = sums[i];
    for (int k = 1; k < teams; ++k) v += sums[k * 2 * n.H + i];
    a.partial[static_cast<long long>(blockIdx.x) * 2 * n.H + i] = v;
  }
}

// The same for rows too long for a thread's registers: read from memory twice (the
// next ones fetched to L2 meanwhile), sums in shared memory, a thread's channels its
// own, [pre, y][first, second four of a word][words].
template <bool kRes32>
__global__ void __launch_bounds__(kRingThreads, 1) k_block_norm_backward_long(const BlockNormBackwardArgs a) {
  extern __shared__ float4 own[];
  __shared__ float part[2][3][kRingWarps];
  after_previous();
  const BlockNormArgs& n = a.n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = n.H >> 3;
  const float inv_h = 1.0f / static_cast<float>(n.H);
  const bool pre = a.grad_x != nullptr, post = a.need_y && n.post;
  for (int i = tid; i < 4 * words; i += kRingThreads) own[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __syncthreads();
  auto take = [&](const float4* o, float* v) {
    const float4 a = o[0], b = o[words];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  };
  auto put = [&](float4* o, const float* v) {
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[words] = make_float4(v[4], v[5], v[6], v[7]);
  };
  int turn = 0;
  for (long long t = blockIdx.x; t < n.T; t += gridDim.x) {
    const long long row = t * words;
    if (n.mask && !n.mask[t]) {
      const float zero[8] = {};
      for (int c = tid; c < words; c += kRingThreads) {
        if (a.grad_residual) store8(a.grad_residual, kRes32, row + c, zero);
        if (a.grad_y) store8(a.grad_y, false, row + c, zero);
        if (a.grad_gate && n.gate_per_token) store8(a.grad_gate, false, row + c, zero);
      }
      continue;
    }
    if (tid == 0 && t + gridDim.x < n.T) {
      // the block's next rows on their way to L2
      const long long next = (t + gridDim.x) * n.H;
      constexpr int kR = kRes32 ? 4 : 2;
      if (a.grad_new) prefetch_l2_bulk(static_cast<const char*>(a.grad_new) + next * kR, n.H * kR);
      if (pre) prefetch_l2_bulk(static_cast<const char*>(n.new_residual) + next * kR, n.H * kR);
      if (pre) prefetch_l2_bulk(static_cast<const uint16_t*>(a.grad_x) + next, n.H * 2);
      if (a.need_y) prefetch_l2_bulk(static_cast<const uint16_t*>(n.y) + next, n.H * 2);
      if (n.gate_per_token) prefetch_l2_bulk(static_cast<const uint16_t*>(n.gate) + next, n.H * 2);
    }
    const float r1 = post ? n.rstd[t] : 1.0f, r2 = pre ? n.rstd[n.T + t] : 0.0f;
    float m1 = 0.0f, m2 = 0.0f;
    // word c: g = grad_h + rstd2 a, hn, x, yn, q = scale gate post, u the token's gate
    auto fetch = [&](int c, float* g, float* hn, float* x, float* w, float* y, float* q, float* u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = hn[j] = x[j] = w[j] = y[j] = 0.0f, q[j] = n.scale, u[j] = 1.0f;
      if (a.grad_new) load8(a.grad_new, kRes32, row + c, g);
      if (pre) {
        load8(n.new_residual, kRes32, row + c, hn);
        load8(a.grad_x, false, row + c, x);
        load8(n.pre, n.weight32, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) hn[j] *= r2, g[j] = fmaf(r2 * x[j], w[j], g[j]);
      }
      float v[8];
      if (a.need_y) {
        load8(n.y, false, row + c, y);
        if (n.post) load8(n.post, n.weight32, c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[j] *= r1;
          if (n.post) q[j] *= v[j];
        }
      }
      if (n.gate) {
        load8(n.gate, n.weight32 && !n.gate_per_token, n.gate_per_token ? row + c : c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) (n.gate_per_token ? u : q)[j] *= v[j];
      }
    };
    if (pre || post) {
      float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
      for (int c = tid; c < words; c += kRingThreads) {
        float g[8], hn[8], x[8], w[8], y[8], q[8], u[8];
        fetch(c, g, hn, x, w, y, q, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float b = q[j] * u[j] * y[j];
          s1 = fmaf(x[j] * w[j], hn[j], s1);
          s2 = fmaf(b, g[j], s2);
          s3 = fmaf(b, hn[j], s3);
        }
      }
      s1 = warp_sum(s1), s2 = warp_sum(s2), s3 = warp_sum(s3);
      if (lane == 0) part[turn][0][warp] = s1, part[turn][1][warp] = s2, part[turn][2][warp] = s3;
      __syncthreads();
      s1 = s2 = s3 = 0.0f;
#pragma unroll
      for (int w = 0; w < kRingWarps; ++w) s1 += part[turn][0][w], s2 += part[turn][1][w], s3 += part[turn][2][w];
      turn ^= 1;
      m1 = s1 * inv_h * r2;
      if (post) m2 = inv_h * fmaf(-m1, s3, s2);
    }
    for (int c = tid; c < words; c += kRingThreads) {
      float g[8], hn[8], x[8], w[8], y[8], q[8], u[8], dg[8];
      fetch(c, g, hn, x, w, y, q, u);
      float sum[8];
      if (a.grad_pre) {
        take(own + c, sum);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = fmaf(x[j], hn[j], sum[j]);
        put(own + c, sum);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = fmaf(-hn[j], m1, g[j]);
      if (a.sum_y) take(own + 2 * words + c, sum);
      if (a.grad_residual) store8(a.grad_residual, kRes32, row + c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = g[j] * y[j];
        dg[j] = q[j] * v;
        if (a.sum_y) sum[j] = fmaf(u[j], v, sum[j]);
        g[j] = r1 * fmaf(-y[j], m2, q[j] * u[j] * g[j]);
      }
      if (a.sum_y) put(own + 2 * words + c, sum);
      if (a.grad_gate && n.gate_per_token) store8(a.grad_gate, false, row + c, dg);
      if (a.grad_y) store8(a.grad_y, false, row + c, g);
    }
  }
  for (int c = tid; c < words; c += kRingThreads)
    for (int k = 0; k < 2; ++k)
      if (k == 0 ? a.grad_pre != nullptr : a.sum_y) {
        float v[8];
        take(own + 2 * k * words + c, v);
        store8(a.partial + (static_cast<long long>(blockIdx.x) * 2 + k) * n.H, true, c, v);
      }
}

// Sums of the blocks' partial [block][2][H], 32 runs of blocks side by side:
// pre's gradient, and sum(gh yn), which times scale and the gate is post's
// gradient and times scale and post the gate's.
constexpr int kRuns = 32, kRunWords = 256 / kRuns;
__global__ void __launch_bounds__(256) k_block_norm_sums(const BlockNormBackwardArgs a, int blocks) {
  __shared__ float4 runs[kRuns][kRunWords];
  after_previous();
  const BlockNormArgs& n = a.n;
  const int word = threadIdx.x % kRunWords, run = threadIdx.x / kRunWords;
  const int i = (blockIdx.x * kRunWords + word) * 4;
  const bool on = i < n.H && (blockIdx.y ? a.sum_y : a.grad_pre != nullptr);
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (on) {
#pragma unroll 8
    for (int b = run; b < blocks; b += kRuns) {
      const float4 v = *reinterpret_cast<const float4*>(a.partial + (static_cast<long long>(b) * 2 + blockIdx.y) * n.H + i);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
  }
  runs[run][word] = s;
  __syncthreads();
  if (run || !on) return;
#pragma unroll 8
  for (int r = 1; r < kRuns; ++r) {
    const float4 v = runs[r][word];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  if (blockIdx.y == 0) {
    *reinterpret_cast<float4*>(a.grad_pre + i) = s;
    return;
  }
  const float v[4] = {s.x, s.y, s.z, s.w};
  auto weight = [&](const void* p, int at) {
    return n.weight32 ? static_cast<const float*>(p)[at] : bf16_lo(static_cast<const uint16_t*>(p)[at]);
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float scaled = n.scale * v[j];
    if (a.grad_post) a.grad_post[i + j] = n.gate && !n.gate_per_token ? scaled * weight(n.gate, i + j) : scaled;
    if (a.grad_gate && !n.gate_per_token) static_cast<float*>(a.grad_gate)[i + j] = n.post ? scaled * weight(n.post, i + j) : scaled;
  }
}

namespace {

// Shared memory for rings on the current device.
cudaError_t ring_room(int* room) {
  int device = 0, smem = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
  *room = smem - static_cast<int>((sizeof(RingShared) + kRingAlign - 1) / kRingAlign * kRingAlign);
  return e;
}

// a / b rounded up, for every a that an int holds.
int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Warps that hold a row.
int row_warps(int H, int words_each) { return (H / 8 + 32 * words_each - 1) / (32 * words_each); }

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, bool res32, int sms, cudaStream_t stream) {
  cudaError_t e;
  if (a.H <= kRingHidden) {
    const bool y = a.y != nullptr, token = y && a.gate_per_token;
    using Kernel = void (*)(BlockNormArgs, int, int);
    static const Kernel kernels[12] = {
        k_block_norm<false, false, false, false>, k_block_norm<false, true, false, false>, k_block_norm<false, true, true, true>,
        k_block_norm<true, false, false, false>,  k_block_norm<true, true, false, false>,  k_block_norm<true, true, true, true>,
        k_block_norm<false, false, false, true>,  k_block_norm<false, true, false, true>,  k_block_norm<false, true, true, true>,
        k_block_norm<true, false, false, true>,   k_block_norm<true, true, false, true>,   k_block_norm<true, true, true, true>};
    const int which = (a.mask ? 6 : 0) + res32 * 3 + y + token;
    const Kernel kernel = kernels[which];
    static std::atomic<unsigned long long> ready[12];  // devices set up, a bit each
    int room = 0;
    if ((e = set_up_kernel(reinterpret_cast<const void*>(kernel), ready[which], 0)) != cudaSuccess ||
        (e = ring_room(&room)) != cudaSuccess)
      return e;
    const int bytes = a.H * ((res32 ? 4 : 2) + (y ? 2 : 0) + (token ? 2 : 0));
    const int warps = row_warps(a.H, kWordsEach), per_sm = ceil_div(a.T, sms);
    int teams = kRingWarps / warps;
    if (teams > per_sm) teams = per_sm;
    if (teams > room / (2 * bytes)) teams = room / (2 * bytes);
    int stages = room / (bytes * teams);
    if (stages > kMaxStages) stages = kMaxStages;
    const int most = ceil_div(a.T, teams);
    return launch_early(kernel, 1, dim3(sms < most ? sms : most), dim3(teams * warps * 32), bytes * teams * stages, stream,
                        a, warps, stages);
  }
  using Kernel = void (*)(BlockNormArgs);
  static const Kernel kernels[2][2] = {{k_block_norm_long<3, false>, k_block_norm_long<4, false>},
                                       {k_block_norm_long<3, true>, k_block_norm_long<4, true>}};
  static_assert(kRingHidden >= 2 * 8 * kRingThreads && kBlockNormMaxHidden <= 4 * 8 * kRingThreads, "");
  return launch_early(kernels[res32][a.H > 3 * 8 * kRingThreads], 1, dim3(sms < a.T ? sms : a.T), dim3(kRingThreads), 0,
                      stream, a);
}

namespace {

using Backward = void (*)(BlockNormBackwardArgs, int, int);
template <int kWarps, int kWords, bool kRes32>
Backward backward_kernel(bool pre, bool y, bool token) {
  constexpr int kThreads = 32 * kWarps, kGated = kRes32 ? kRingThreads : kThreads;
  static const Backward kernels[8] = {
      k_block_norm_backward<kThreads, kWords, kRes32, false, false, false>, k_block_norm_backward<kGated, kWords, kRes32, false, false, true>,
      k_block_norm_backward<kThreads, kWords, kRes32, false, true, false>,  k_block_norm_backward<kGated, kWords, kRes32, false, true, true>,
      k_block_norm_backward<kThreads, kWords, kRes32, true, false, false>,  k_block_norm_backward<kGated, kWords, kRes32, true, false, true>,
      k_block_norm_backward<kThreads, kWords, kRes32, true, true, false>,   k_block_norm_backward<kGated, kWords, kRes32, true, true, true>};
  return kernels[pre * 4 + y * 2 + token];
}

}  // namespace

cudaError_t launch_block_norm_backward(const BlockNormBackwardArgs& args, bool res32, int sms, cudaStream_t stream) {
  BlockNormBackwardArgs a = args;
  const bool token = a.n.gate && a.n.gate_per_token, block = a.grad_y || a.grad_gate || a.grad_post;
  a.need_y = a.grad_gate || a.grad_post || (a.grad_y && a.n.post);
  a.sum_y = a.grad_post || (a.grad_gate && !token);
  int blocks = sms < kBlockNormMaxBlocks ? sms : kBlockNormMaxBlocks;
  cudaError_t e;
  // A row's words over as few warps as hold them, and as many teams of them as fill
  // a block and leave each two stages of all that a row can have (so that no sum's
  // order depends on which gradients are asked for), unless SMs would have no rows.
  const bool gate = token && block;
  const int r = res32 ? 4 : 2;
  const int all = a.n.H * (2 * r + 4 + (token ? 2 : 0)), bytes = a.n.H * ((a.grad_new ? r : 0) + (a.grad_x ? r + 2 : 0) + (a.need_y ? 2 : 0) + (gate ? 2 : 0));
  int room = 0;
  if ((e = ring_room(&room)) != cudaSuccess) return e;
  if (a.n.H <= kRingHidden && 2 * all <= room) {
    // One word a thread (16 warps of 128 registers) where that fills 15 warps or more, and
    // for fp32 residuals wherever it holds the row: 8192 x 4096 bf16 77 us instead of 84, fp32
    // 99 instead of 122; 2048 fp32 55 instead of 62; 2560 (10 warps) bf16 62 instead of 57.
    const int single = row_warps(a.n.H, 1);
    const bool one = single <= kRingWarps && (res32 || kRingWarps / single * single >= kRingWarps - 1);
    const int warps = one ? single : row_warps(a.n.H, kWordsEach), per_sm = ceil_div(a.n.T, sms);
    const bool wide = one || warps > kNarrowWarps;
    int teams = (wide ? kRingWarps : kNarrowWarps) / warps;
    if (teams > per_sm) teams = per_sm;
    if (teams > room / (2 * all)) teams = room / (2 * all);
    int stages = bytes ? room / (bytes * teams) : 2;
    if (stages > kMaxStages) stages = kMaxStages;
    const int sums = teams > 1 ? 8 * a.n.H * teams : 0;
    const int need = bytes * teams * stages > sums ? bytes * teams * stages : sums;
    auto pick = one    ? (res32 ? backward_kernel<kRingWarps, 1, true> : backward_kernel<kRingWarps, 1, false>)
                : wide ? (res32 ? backward_kernel<kRingWarps, kWordsEach, true> : backward_kernel<kRingWarps, kWordsEach, false>)
                       : (res32 ? backward_kernel<kNarrowWarps, kWordsEach, true> : backward_kernel<kNarrowWarps, kWordsEach, false>);
    auto kernel = pick(a.grad_x != nullptr, a.need_y, gate);
    static std::atomic<unsigned long long> ready[48];  // devices set up, a bit each
    const int which = (one + wide) * 16 + res32 * 8 + (a.grad_x != nullptr) * 4 + a.need_y * 2 + gate;
    if ((e = set_up_kernel(reinterpret_cast<const void*>(kernel), ready[which], 0)) != cudaSuccess) return e;
    const int most = ceil_div(a.n.T, teams);
    if (blocks > most) blocks = most;
    e = launch_early(kernel, 1, dim3(blocks), dim3(teams * warps * 32), need, stream, a, warps, stages);
  } else {
    auto kernel = res32 ? k_block_norm_backward_long<true> : k_block_norm_backward_long<false>;
    static std::atomic<unsigned long long> ready[2];
    if ((e = set_up_kernel(reinterpret_cast<const void*>(kernel), ready[res32], 0)) != cudaSuccess) return e;
    if (blocks > a.n.T) blocks = a.n.T;
    e = launch_early(kernel, 1, dim3(blocks), dim3(kRingThreads), sizeof(float) * 2 * a.n.H, stream, a);
  }
  if (e != cudaSuccess || !(a.grad_pre || a.sum_y)) return e;
  return launch_early(k_block_norm_sums, 1, dim3((a.n.H + 4 * kRunWords - 1) / (4 * kRunWords), 2), dim3(256), 0, stream, a, blocks);
}

}  // namespace ep
