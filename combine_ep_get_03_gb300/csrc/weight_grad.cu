// Weight gradient of the experts' product from 8-bit rows:
//   dw[e, n, k] = sum over the rows r of group e of dy[r, n] x[r, k],
// both e4m3 with a scale for every 128 channels of a row.
//
// The contraction runs over rows, and both scales change with the row, so they
// cannot be taken out of the sum: the operands are widened to f16 on the way
// to shared memory and multiplied by f16 tensor-core instructions with fp32
// accumulation.  A 128-column tile of dy lies in one scale group, so dy enters
// as its codes (exact in f16) and x carries the product of both scales,
// divided by a power of two that brings the tile's largest below one and is
// put back on the fp32 sums.  That costs x two roundings to 11 bits, an eighth
// of the rounding of the bf16 result.
//
// Tile 128 (n) x 256 (k), 64 rows a stage.  Two teams of eight warps take
// every other stage: they fetch e4m3 rows a turn ahead (also across tiles),
// widen and store them with the 128-byte swizzle, rows along the long axis (both operands "MN major", so nothing is
// transposed); one warp issues four MMAs a stage; four more write the previous
// tile from the other TMEM accumulator; one looks up the next tile's largest
// scale.  Rows past the group's end enter as zeros.
#include "ep_internal.h"
#include "experts.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

constexpr int kTileN = 128, kTileK = 256, kRows = 64;
constexpr int kStages = 4;
constexpr int kChunkBytes = kRows * 128;  // 64 columns of f16
constexpr int kStageBytes = (kTileN + kTileK) / 64 * kChunkBytes;
constexpr int kTeams = 2, kTeamWarps = 8, kLoadWarps = kTeams * kTeamWarps, kStoreWarps = 4;
constexpr int kMmaWarp = kLoadWarps + kStoreWarps, kScaleWarp = kMmaWarp + 1;
constexpr int kThreads = (kScaleWarp + 1) * 32;
constexpr uint32_t kTmemColumns = 512;
constexpr int kExponents = 4;  // tiles whose exponents are kept

struct Shared {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], exp_full[kExponents], exp_empty[kExponents];
  uint32_t tmem;
  int quit;
  int exponent[kExponents][2];
};

// First row and row count of every group, in shared memory.
struct Group {
  int row, rows;
};

// The block's tiles that have rows, one after another.
struct Walk {
  const Group* groups;
  int tiles_n, tiles_k;
  unsigned t, tiles;
  int group, n, k, rows;
  __device__ __forceinline__ void set() {
    const unsigned row = t / static_cast<unsigned>(tiles_k);
    k = static_cast<int>(t - row * tiles_k);
    group = static_cast<int>(row / static_cast<unsigned>(tiles_n));
    n = static_cast<int>(row - group * tiles_n);
    rows = groups[group].rows;
  }
  __device__ __forceinline__ bool settle() {  // at t or after it
    for (; t < tiles; t += gridDim.x) {
      set();
      if (rows) return true;
    }
    return false;
  }
  __device__ __forceinline__ bool next() {
    t += gridDim.x;
    return settle();
  }
  __device__ __forceinline__ int blocks() const { return (rows + kRows - 1) / kRows; }
  __device__ __forceinline__ long long row() const { return groups[group].row; }
};

// A block of rows of a walk: block b of the used-th tile that has rows.
struct Cursor {
  Walk w;
  int b, blocks;
  uint32_t used;
  bool on;
  __device__ __forceinline__ void begin(const Walk& walk) {
    w = walk;
    b = 0;
    used = 0;
    on = w.settle();
    blocks = on ? w.blocks() : 0;
  }
  __device__ __forceinline__ void step() {
    if (on && ++b == blocks) {
      on = w.next();
      blocks = on ? w.blocks() : 0;
      b = 0;
      ++used;
    }
  }
};

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

// Four e4m3 codes as two f16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t* lo, uint32_t* hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(*lo), "=r"(*hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" : : "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 codes to f16, at the two shared-memory addresses of their 16-byte units.
__device__ __forceinline__ void store_chunk(uint32_t lo, uint32_t hi, const uint4& q, uint32_t scale, bool scaled) {
  uint32_t h[8];
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e4m3x4_to_f16(w[i], &h[2 * i], &h[2 * i + 1]);
    if (scaled) h[2 * i] = mul_f16x2(h[2 * i], scale), h[2 * i + 1] = mul_f16x2(h[2 * i + 1], scale);
  }
  sts128(lo, h[0], h[1], h[2], h[3]);
  sts128(hi, h[4], h[5], h[6], h[7]);
}

// A load that stays where it is written, far ahead of its use.
__device__ __forceinline__ uint4 ld_ahead(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_ahead_f32(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// One thread's part of 64 rows: of one row, chunks c, c + 4 of dy and c, c + 4,
// c + 8, c + 12 of x (c = thread mod 4), and the scales of both halves of x.
struct Fetched {
  uint4 dy[2], x[4];
  float y_scale, x_scale[2];
};

}  // namespace

__global__ void __launch_bounds__(kThreads, 1) k_weight_grad(const WeightGradArgs p) {
  extern __shared__ unsigned char raw[];
  unsigned char* stages = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Shared& s = *reinterpret_cast<Shared*>(stages + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* quit = &s.quit;
  int* err = p.groups.err;
  Group* groups = reinterpret_cast<Group*>(&s + 1);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s.full[i], kTeamWarps), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], kStoreWarps);
    for (int i = 0; i < kExponents; ++i) mbar_init(&s.exp_full[i], 1), mbar_init(&s.exp_empty[i], kStoreWarps);
    s.quit = 0;
    mbar_init_fence();
  }
  if (warp == kMmaWarp) tmem_alloc(&s.tmem, kTmemColumns);
  for (int g = threadIdx.x; g < p.groups.G; g += kThreads) {
    long long start;
    groups[g].rows = group_span(p.groups, g, &start, blockIdx.x == 0);
    groups[g].row = static_cast<int>(start);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem;
  Walk w;
  w.groups = groups;
  w.tiles_n = p.N / kTileN;
  w.tiles_k = (p.K + kTileK - 1) / kTileK;
  w.tiles = static_cast<unsigned>(p.groups.G) * w.tiles_n * w.tiles_k;
  w.t = blockIdx.x;

  if (warp < kLoadWarps) {
    const int team = warp / kTeamWarps, tid = threadIdx.x % (kTeamWarps * 32);
    const int my_row = tid >> 2, chunk = tid & 3;
    // Row my_row, chunk c = chunk + 4 j of an operand lies in 64-channel block j
    // at swizzled units 2 chunk and 2 chunk + 1.  A phase of a warp's 16-byte
    // stores covers two rows, whose units are the even and the odd ones: no
    // bank conflict.
    const uint32_t line = smem_u32(stages) + my_row * 128;
    const uint32_t unit_lo = line + (((2 * chunk) ^ (my_row & 7)) << 4);
    const uint32_t unit_hi = line + (((2 * chunk + 1) ^ (my_row & 7)) << 4);
    Cursor now, next;  // the team's block and the one it fetches
    now.begin(w);
    if (team) now.step();
    next = now;
    // what the fetched tile's block 0 would read, and steps from block to block
    const unsigned char *dy = nullptr, *x = nullptr;
    const float *dy_scale = nullptr, *x_scale = nullptr;
    const long long dy_step = static_cast<long long>(kRows) * p.N, x_step = static_cast<long long>(kRows) * p.K;
    const long long dys_step = kRows * p.dy.row_stride, xs_step = kRows * p.x.row_stride;
    bool second = false;
    auto aim = [&]() {
      const long long r = next.w.row() + my_row;
      dy = p.dy.data + r * p.N + next.w.n * kTileN + chunk * 16 + next.b * dy_step;
      x = p.x.data + r * p.K + next.w.k * kTileK + chunk * 16 + next.b * x_step;
      dy_scale = p.dy.scale(r, next.w.n) + next.b * dys_step;
      x_scale = p.x.scale(r, next.w.k * 2) + next.b * xs_step;
      second = next.w.k * 2 + 1 < (p.K >> 7);
    };
    auto fetch = [&](Fetched& d) {
      const bool on = next.b * kRows + my_row < next.w.rows;
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) d.dy[j] = on ? ld_ahead(dy + j * 64) : zero;
#pragma unroll
      for (int j = 0; j < 4; ++j) d.x[j] = on && (j < 2 || second) ? ld_ahead(x + j * 64) : zero;
      d.y_scale = on ? ld_ahead_f32(dy_scale) : 0.0f;
      d.x_scale[0] = on ? ld_ahead_f32(x_scale) : 0.0f;
      d.x_scale[1] = on && second ? ld_ahead_f32(x_scale + p.x.group_stride) : 0.0f;
    };
    auto advance = [&]() {
      if (next.b + kTeams < next.blocks) {
        next.b += kTeams;
        dy += kTeams * dy_step;
        x += kTeams * x_step;
        dy_scale += kTeams * dys_step;
        x_scale += kTeams * xs_step;
      } else {
        for (int i = 0; i < kTeams; ++i) next.step();
        if (next.on) aim();
      }
    };
    if (next.on) aim();
    Fetched d;
    if (next.on) fetch(d);
    uint32_t tile = ~0u;  // whose exponents `down` holds
    float down[2] = {1.0f, 1.0f};
    for (uint32_t it = team; now.on; it += kTeams) {
      const int st = it % kStages;
      bool ok = true;
      if (now.used != tile) {
        tile = now.used;
        const int e = tile % kExponents;
        ok = wait_or_quit(&s.exp_full[e], (tile / kExponents) & 1, quit, err);
        down[0] = power_of_two(-s.exponent[e][0]);
        down[1] = power_of_two(-s.exponent[e][1]);
      }
      if (it >= kStages) ok = ok && wait_or_quit(&s.empty[st], ((it / kStages) & 1) ^ 1, quit, err);
      if (!__all_sync(kFullMask, ok)) break;
      const uint32_t lo = unit_lo + st * kStageBytes, hi = unit_hi + st * kStageBytes;
#pragma unroll
      for (int j = 0; j < 2; ++j) store_chunk(lo + j * kChunkBytes, hi + j * kChunkBytes, d.dy[j], 0u, false);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float sc = d.y_scale * d.x_scale[j >> 1] * down[j >> 1];
        uint32_t h;
        asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(h) : "f"(sc));
        store_chunk(lo + (2 + j) * kChunkBytes, hi + (2 + j) * kChunkBytes, d.x[j], h, true);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.full[st]);
      advance();
      if (next.on) fetch(d);
      now = next;
    }
  } else if (warp == kScaleWarp) {
    // the largest scale of each half of the tiles to come: 2^e above it
    uint32_t used = 0;
    for (bool on = w.settle(); on; on = w.next(), ++used) {
      const int e = used % kExponents;
      if (used >= kExponents &&
          !__all_sync(kFullMask, wait_or_quit(&s.exp_empty[e], ((used / kExponents) & 1) ^ 1, quit, err)))
        break;
      const bool second = w.k * 2 + 1 < (p.K >> 7);
      const float* ys = p.dy.scale(w.row(), w.n);
      const float* xs = p.x.scale(w.row(), w.k * 2);
      float m[2] = {0.0f, 0.0f};
#pragma unroll 8
      for (int r = lane; r < w.rows; r += 32) {
        const float y = ys[r * p.dy.row_stride];
        m[0] = fmaxf(m[0], fabsf(y * xs[r * p.x.row_stride]));
        if (second) m[1] = fmaxf(m[1], fabsf(y * xs[r * p.x.row_stride + p.x.group_stride]));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        m[0] = fmaxf(m[0], __shfl_xor_sync(kFullMask, m[0], d));
        m[1] = fmaxf(m[1], __shfl_xor_sync(kFullMask, m[1], d));
      }
      if (lane == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // a scale without a finite largest is used as it is
          const int x = m[h] > 0.0f && m[h] < 3.0e38f ? ilogbf(m[h]) + 1 : 0;
          s.exponent[e][h] = max(-100, min(100, x));
        }
        mbar_arrive(&s.exp_full[e]);
      }
      __syncwarp();
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t desc = mma_desc(kTileN, kTileK, true);
    const uint64_t first = smem_desc(smem_u32(stages), kChunkBytes, 1024);
    uint32_t it = 0, used = 0;
    bool ok = true;
    for (bool on = w.settle(); ok && on; on = w.next()) {
      const int ac = used & 1, blocks = w.blocks();
      ok = __all_sync(kFullMask, used < 2 || wait_or_quit(&s.acc_empty[ac], ((used >> 1) & 1) ^ 1, quit, err));
      if (!ok) break;
      for (int b = 0; b < blocks; ++b, ++it) {
        const int st = it % kStages;
        ok = __all_sync(kFullMask, wait_or_quit(&s.full[st], (it / kStages) & 1, quit, err));
        if (!ok) break;
        tmem_fence_after();
        if (elect_one()) {
          // descriptors count 16-byte units; an MMA takes 16 rows of 128 bytes
          const uint64_t dy = first + st * (kStageBytes >> 4), x = dy + (kTileN / 64 * kChunkBytes >> 4);
          const int steps = (min(kRows, w.rows - b * kRows) + 15) >> 4;
#pragma unroll
          for (int j = 0; j < kRows / 16; ++j)
            if (j < steps) mma_f16(tmem + ac * kTileK, dy + 128 * j, x + 128 * j, desc, b > 0 || j > 0);
          mma_commit(&s.empty[st]);
        }
        __syncwarp();
      }
      // also after a wait that gave up: what was issued ends before TMEM goes back
      if (elect_one()) mma_commit(&s.acc_full[ac]);
      __syncwarp();
      ++used;
    }
    for (uint32_t i = used < 2 ? 0 : used - 2; i < used; ++i) {
      int none = 0;
      wait_or_quit(&s.acc_full[i & 1], (i >> 1) & 1, &none, err);
    }
  } else {
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const bool wide = (reinterpret_cast<uintptr_t>(p.dw) & 31) == 0;
    uint32_t used = 0;
    for (; w.t < w.tiles; w.t += gridDim.x) {
      w.set();
      uint16_t* o = p.dw + (static_cast<long long>(w.group) * p.N + w.n * kTileN + quarter * 32 + lane) * p.K + w.k * kTileK;
      const int columns = min(kTileK, p.K - w.k * kTileK);
      if (w.rows == 0) {
        const uint32_t zero[8] = {};
        for (int q = 0; q < columns; q += 16) store32(o + q, zero, wide);
        continue;
      }
      const int ac = used & 1, e = used % kExponents;
      if (!__all_sync(kFullMask, wait_or_quit(&s.exp_full[e], (used / kExponents) & 1, quit, err) &&
                                     wait_or_quit(&s.acc_full[ac], (used >> 1) & 1, quit, err)))
        break;
      tmem_fence_after();
      const float up[2] = {power_of_two(s.exponent[e][0]), power_of_two(s.exponent[e][1])};
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.exp_empty[e]);
#pragma unroll
      for (int q = 0; q < kTileK / 32; ++q) {
        uint32_t v[32];
        tmem_load32(lanes + ac * kTileK + q * 32, v);
        tmem_load_wait(v);
        if (q == kTileK / 32 - 1) {
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.acc_empty[ac]);
        }
        const float f = up[q >> 2];
        if (q * 32 < columns) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              x[j] = pack_bf16x2(__uint_as_float(v[h * 16 + 2 * j]) * f, __uint_as_float(v[h * 16 + 2 * j + 1]) * f);
            store32(o + q * 32 + h * 16, x, wide);
          }
        }
      }
      ++used;
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tmem_fence_after();
    tmem_free(tmem, kTmemColumns);
  }
}

cudaError_t launch_weight_grad(const WeightGradArgs& p, int sms, cudaStream_t stream) {
  const size_t smem = 1024 + static_cast<size_t>(kStages) * kStageBytes + sizeof(Shared) + sizeof(Group) * p.groups.G;
  static std::atomic<unsigned long long> ready;  // devices set up, a bit each
  const cudaError_t e = set_up_kernel(reinterpret_cast<const void*>(k_weight_grad), ready, 0);
  if (e != cudaSuccess) return e;
  return launch_kernel(k_weight_grad, dim3(sms), dim3(kThreads), smem, stream, p);
}

}  // namespace ep
