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
// Tile 128 (n) x 256 (k).  Eight warps fetch e4m3 rows 64 at a time, widen
// and store them with the 128-byte swizzle, rows along the long axis (both
// operands "MN major", so nothing is transposed); one thread issues four MMAs
// for them; four more warps write the previous tile from the other TMEM
// accumulator.  Rows past the group's end enter as zeros.
#include "ep_internal.h"
#include "experts.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

constexpr int kTileN = 128, kTileK = 256, kRows = 64;
constexpr int kStages = 4;
constexpr int kChunkBytes = kRows * 128;  // 64 columns of f16
constexpr int kStageBytes = (kTileN + kTileK) / 64 * kChunkBytes;
constexpr int kLoadWarps = 8, kStoreWarps = 4;
constexpr int kThreads = (kLoadWarps + kStoreWarps + 1) * 32;
constexpr uint32_t kTmemColumns = 512;
constexpr int kExponents = 8;  // tiles whose exponents are kept: stages + accumulators + 1, rounded up

struct Shared {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], max_full;
  uint32_t tmem;
  int quit;
  float max_part[2][kLoadWarps][2];
  int exponent[kExponents][2];
};

struct Tile {
  int group, n, k, rows;
  long long row;
};

__device__ __forceinline__ Tile tile_at(const GroupArgs& a, int tiles_n, int tiles_k, long long t, bool report) {
  Tile c;
  const long long per = static_cast<long long>(tiles_n) * tiles_k;
  c.group = static_cast<int>(t / per);
  const int local = static_cast<int>(t % per);
  c.n = local / tiles_k;
  c.k = local % tiles_k;
  c.rows = group_span(a, c.group, &c.row, report);
  return c;
}

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
__device__ __forceinline__ void sts128(unsigned char* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" : : "r"(smem_u32(p)), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 codes of row r, 16-channel chunk c of an operand, to its f16 tile.  A
// phase of a warp's 16-byte stores covers two rows of one 64-channel block,
// whose swizzled units are the even and the odd ones: no bank conflict.
__device__ __forceinline__ void store_chunk(unsigned char* tile, int r, int c, const uint4& q, uint32_t scale, bool scaled) {
  uint32_t h[8];
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e4m3x4_to_f16(w[i], &h[2 * i], &h[2 * i + 1]);
    if (scaled) h[2 * i] = mul_f16x2(h[2 * i], scale), h[2 * i + 1] = mul_f16x2(h[2 * i + 1], scale);
  }
  unsigned char* line = tile + (c >> 2) * kChunkBytes + r * 128;
  const int u = (c & 3) * 2, x = r & 7;
  sts128(line + ((u ^ x) << 4), h[0], h[1], h[2], h[3]);
  sts128(line + (((u + 1) ^ x) << 4), h[4], h[5], h[6], h[7]);
}

// One thread's part of 64 rows, all of one row: chunks c, c + 4 of dy and
// c, c + 4, c + 8, c + 12 of x (c = thread mod 4), and the row's scales.
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
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s.full[i], kLoadWarps), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], kStoreWarps);
    mbar_init(&s.max_full, kLoadWarps);
    s.quit = 0;
    mbar_init_fence();
  }
  if (warp == kLoadWarps + kStoreWarps) tmem_alloc(&s.tmem, kTmemColumns);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem;
  const int tiles_n = p.N / kTileN, tiles_k = (p.K + kTileK - 1) / kTileK;
  const long long tiles = static_cast<long long>(p.groups.G) * tiles_n * tiles_k;

  if (warp < kLoadWarps) {
    const int tid = threadIdx.x;
    const int my_row = tid >> 2, chunk = tid & 3;
    uint32_t it = 0, used = 0;                        // stages filled, tiles with rows
    bool ok = true;
    for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const Tile c = tile_at(p.groups, tiles_n, tiles_k, t, blockIdx.x == 0 && tid == 0);
      if (c.rows == 0) continue;
      const int group0 = c.k * 2, groups = p.K >> 7;
      const bool second = group0 + 1 < groups;
      const unsigned char* dy0 = p.dy.data + (c.row + my_row) * p.N + c.n * kTileN + chunk * 16;
      const unsigned char* x0 = p.x.data + (c.row + my_row) * p.K + c.k * kTileK + chunk * 16;
      const float* dy_scale = p.dy.scale(c.row + my_row, c.n);
      const float* x_scale = p.x.scale(c.row + my_row, group0);
      const int blocks = (c.rows + kRows - 1) / kRows;
      auto fetch = [&](int b, Fetched& f) {
        const long long r = static_cast<long long>(b) * kRows;
        const bool on = my_row + r < c.rows;
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 2; ++j) f.dy[j] = on ? ld_stream(dy0 + r * p.N + j * 64) : zero;
#pragma unroll
        for (int j = 0; j < 4; ++j) f.x[j] = on && (j < 2 || second) ? ld_stream(x0 + r * p.K + j * 64) : zero;
        f.y_scale = on ? dy_scale[r * p.dy.row_stride] : 0.0f;
        f.x_scale[0] = on ? x_scale[r * p.x.row_stride] : 0.0f;
        f.x_scale[1] = on && second ? x_scale[r * p.x.row_stride + p.x.group_stride] : 0.0f;
      };
      Fetched ahead[2];  // two blocks of rows are on their way
      fetch(0, ahead[0]);
      fetch(1, ahead[1]);
      // the largest scale of each half of the tile
      float m0 = 0.0f, m1 = 0.0f;
      for (int r = tid; r < c.rows; r += kLoadWarps * 32) {
        const float y = *p.dy.scale(c.row + r, c.n);
        m0 = fmaxf(m0, fabsf(y * *p.x.scale(c.row + r, group0)));
        if (second) m1 = fmaxf(m1, fabsf(y * *p.x.scale(c.row + r, group0 + 1)));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(kFullMask, m0, d));
        m1 = fmaxf(m1, __shfl_xor_sync(kFullMask, m1, d));
      }
      if (lane == 0) {
        s.max_part[used & 1][warp][0] = m0;
        s.max_part[used & 1][warp][1] = m1;
        mbar_arrive(&s.max_full);
      }
      ok = __all_sync(kFullMask, wait_or_quit(&s.max_full, used & 1, quit, err));
      if (!ok) break;
      float down[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < kLoadWarps; ++w) m = fmaxf(m, s.max_part[used & 1][w][h]);
        // 2^e > m; a scale without a finite largest is used as it is
        int e = m > 0.0f && m < 3.0e38f ? ilogbf(m) + 1 : 0;
        e = max(-100, min(100, e));
        if (tid == 0) s.exponent[used % kExponents][h] = e;
        down[h] = power_of_two(-e);
      }
      auto block = [&](int b, Fetched& f) {
        const int st = it % kStages;
        if (it >= kStages) {
          ok = __all_sync(kFullMask, wait_or_quit(&s.empty[st], ((it / kStages) & 1) ^ 1, quit, err));
          if (!ok) return;
        }
        unsigned char* dy_tile = stages + st * kStageBytes;
        unsigned char* x_tile = dy_tile + kTileN / 64 * kChunkBytes;
#pragma unroll
        for (int j = 0; j < 2; ++j) store_chunk(dy_tile, my_row, chunk + 4 * j, f.dy[j], 0u, false);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float sc = f.y_scale * f.x_scale[j >> 1] * down[j >> 1];
          uint32_t h;
          asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(h) : "f"(sc));
          store_chunk(x_tile, my_row, chunk + 4 * j, f.x[j], h, true);
        }
        fetch(b + 2, f);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.full[st]);
        ++it;
      };
      for (int b = 0; ok && b < blocks; b += 2) {
        block(b, ahead[0]);
        if (ok && b + 1 < blocks) block(b + 1, ahead[1]);
      }
      ++used;
    }
  } else if (warp == kLoadWarps + kStoreWarps) {
    constexpr uint32_t desc = mma_desc(kTileN, kTileK, true);
    const uint64_t first = smem_desc(smem_u32(stages), kChunkBytes, 1024);
    uint32_t it = 0, used = 0;
    bool ok = true;
    for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const Tile c = tile_at(p.groups, tiles_n, tiles_k, t, false);
      if (c.rows == 0) continue;
      const int ac = used & 1, blocks = (c.rows + kRows - 1) / kRows;
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
          const int steps = (min(kRows, c.rows - b * kRows) + 15) >> 4;
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
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
      const Tile c = tile_at(p.groups, tiles_n, tiles_k, t, false);
      uint16_t* o = p.dw + (static_cast<long long>(c.group) * p.N + c.n * kTileN + quarter * 32 + lane) * p.K + c.k * kTileK;
      const int columns = min(kTileK, p.K - c.k * kTileK);
      if (c.rows == 0) {
        const uint32_t zero[8] = {};
        for (int q = 0; q < columns; q += 16) store32(o + q, zero, wide);
        continue;
      }
      const int ac = used & 1;
      if (!__all_sync(kFullMask, wait_or_quit(&s.acc_full[ac], (used >> 1) & 1, quit, err))) break;
      tmem_fence_after();
      const float up[2] = {power_of_two(s.exponent[used % kExponents][0]), power_of_two(s.exponent[used % kExponents][1])};
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
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              w[j] = pack_bf16x2(__uint_as_float(v[h * 16 + 2 * j]) * f, __uint_as_float(v[h * 16 + 2 * j + 1]) * f);
            store32(o + q * 32 + h * 16, w, wide);
          }
        }
      }
      ++used;
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == kLoadWarps + kStoreWarps) {
    tmem_fence_after();
    tmem_free(tmem, kTmemColumns);
  }
}

cudaError_t launch_weight_grad(const WeightGradArgs& p, int sms, cudaStream_t stream) {
  const size_t smem = 1024 + static_cast<size_t>(kStages) * kStageBytes + sizeof(Shared);
  static std::atomic<unsigned long long> ready;  // devices set up, a bit each
  const cudaError_t e = set_up_kernel(reinterpret_cast<const void*>(k_weight_grad), ready, 0);
  if (e != cudaSuccess) return e;
  return launch_kernel(k_weight_grad, dim3(sms), dim3(kThreads), smem, stream, p);
}

}  // namespace ep
