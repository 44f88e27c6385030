// The experts' products on 4-bit weights, for serving: for a row r of group e
//   y[r, n] = sum_kb sx[r, kb] sum_{k in block kb} x[r, k] c[e, n, k] 2^(s[e, n, k / 32] - 127)
// x e4m3 with a scale for every 128 channels, c e2m1 with an exponent for every
// 32.  Stored as bf16, or (SwiGLU) taken through row_weight silu(gate) up and
// stored as e4m3 with scales.
//
// Few rows are the case that matters, and there the weights' stream is all the
// time: 17 bytes for 32 weights, half of the 8-bit product's.  So the weights
// are the MMA's 128-row operand and the tokens its columns, as few as there are
// rounded up to 16.  TMA spreads the codes to the byte each that the tensor
// cores take beside 8-bit operands, and the exponents are applied inside the
// MMA (their blocks of 512 bytes go from shared memory to TMEM): no instruction
// unpacks or scales a weight.  Every 128 channels have a fresh accumulator, since
// x's scales are arbitrary; the adding warps read it, a lane a weight row, and
// add it to fp32 registers times its column's scale.
//
// Tile 256 weight rows (two halves of 128, in SwiGLU the gate's and the up
// projection's of the same channels) x up to 112 tokens; two accumulators of
// both halves take 448 TMEM columns, the scales the next ones.
#include <cuda.h>

#include <atomic>

#include "ep_internal.h"
#include "experts.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

constexpr int kTileT = kTile4Rows, kBlockK = 128;
constexpr int kChunks = kTileT / 16;
constexpr int kMaxStages = 8, kMaxAcc = 4;
constexpr int kHalfBytes = 128 * kBlockK;  // codes of 128 weight rows, a byte each
constexpr int kHalfLoad = kHalfBytes / 2;  // ... as the transaction counts them
constexpr int kScaleBytes = 512;           // exponents of 128 weight rows
// a stage: both halves, their exponents, the tokens; swizzled operands start at 1024-byte boundaries
constexpr int kTokens = 2 * kHalfBytes + 2 * kScaleBytes;
static_assert(kTokens % 1024 == 0 && 16 * kBlockK % 1024 == 0, "");
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = (kEpilogueWarps + 4) * 32;  // a load, two MMA and a scale warp are the third warpgroup
constexpr int kLaunchRegisters = 168, kEpilogueRegisters = 232, kOtherRegisters = 40;
static_assert(kEpilogueWarps * 32 * kEpilogueRegisters + 4 * 32 * kOtherRegisters <= kThreads * kLaunchRegisters, "");
constexpr uint32_t kTmemColumns = 512;
constexpr uint32_t kWeightScales = 4 * kTileT, kTokenScales = kWeightScales + 16;
static_assert(kTokenScales + 4 <= kTmemColumns, "");
constexpr int kScaleSlots = 16;  // blocks of k whose scales are kept: more than stages and accumulators together
static_assert(kMaxStages + kMaxAcc < kScaleSlots, "");

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[kMaxAcc], acc_empty[kMaxAcc], amax_full[2];
  uint32_t tmem;
  int quit, columns;
  unsigned sums[32];
  alignas(16) float x_scale[kScaleSlots][kTileT];
  float amax[2][2][4][kTileT / 2];  // [tile parity][half][warp][token]
};

struct Tile {
  int group, n;   // group and column tile
  long long row;  // first row
  int rows;       // live rows of the tile
  int columns;    // ... rounded up to 16
};

// Rows of the tiles of a group of `count` rows (the last may have fewer): about
// as many in each, a multiple of 16, which an MMA's columns are.
__device__ __forceinline__ int rows_per_tile(int count, int tiles_m) {
  return tiles_m ? ((count + tiles_m - 1) / tiles_m + 15) & ~15 : 16;
}

__device__ __forceinline__ Tile tile_at(const GroupArgs& a, const unsigned* prefix, int tiles_n, unsigned t) {
  const int g = find_group(prefix, a.G, t / static_cast<unsigned>(tiles_n));
  Tile r;
  long long start;
  const int count = group_span(a, g, &start, false);
  const int tiles_m = (count + kTileT - 1) / kTileT;
  const unsigned local = t - prefix[g] * tiles_n;
  r.group = g;
  r.n = tiles_m ? static_cast<int>(local / static_cast<unsigned>(tiles_m)) : 0;
  const int m = static_cast<int>(local) - r.n * tiles_m;
  const int per = rows_per_tile(count, tiles_m);
  r.row = start + static_cast<long long>(m) * per;
  r.rows = tiles_m ? max(0, min(per, count - m * per)) : 0;
  r.columns = max(16, (r.rows + 15) & ~15);  // an MMA has 16 at least
  return r;
}

}  // namespace

template <bool kSwiglu>
__global__ void __launch_bounds__(kThreads, 1)
    k_grouped_matmul_w4(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                        const Matmul4Args p, uint32_t smem_bytes) {
  extern __shared__ unsigned char raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  unsigned* prefix = reinterpret_cast<unsigned*>(&s + 1);
  unsigned char* stages = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(prefix + p.groups.G + 1) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* quit = &s.quit;
  int* err = p.groups.err;

  if (threadIdx.x == 0) {
    // the loading thread's arrival and one of each of the scale warp's lanes
    for (int i = 0; i < kMaxStages; ++i) mbar_init(&s.full[i], 1 + 32), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < kMaxAcc; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], kEpilogueWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&s.amax_full[i], 4);
    s.quit = 0;
    s.columns = 16;
    mbar_init_fence();
    prefetch_map(&map_x);
    prefetch_map(&map_w);
  }
  if (warp == kEpilogueWarps + 1) tmem_alloc(&s.tmem, kTmemColumns);
  __syncthreads();
  after_previous();
  groups_prefix(p.groups, kTileT, prefix, s.sums,
                [&](int n) { if (n) atomicMax(&s.columns, rows_per_tile(n, (n + kTileT - 1) / kTileT)); });
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem;
  // the tokens' scales inside the MMA are 2^0: theirs are applied behind it
  if (warp < 4) tmem_fill4(tmem + (static_cast<uint32_t>(warp * 32) << 16) + kTokenScales, 0x7f7f7f7fu);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();

  // As many stages as fit beside the largest tile's tokens, and four accumulators
  // where it has few.
  const uint32_t widest = s.columns;
  const uint32_t stage_bytes = kTokens + widest * kBlockK;
  const uint32_t num_stages = min(static_cast<uint32_t>(kMaxStages),
                                  (smem_bytes - static_cast<uint32_t>(stages - raw)) / stage_bytes);
  const uint32_t num_acc = widest * 2 * kMaxAcc <= kWeightScales ? kMaxAcc : 2;

  const int F = p.N >> 1;
  const int blocks_n = (p.N + 127) >> 7;
  const int tiles_n = kSwiglu ? F >> 7 : (blocks_n + 1) >> 1;
  const int blocks_k = p.K / kBlockK;
  const unsigned tiles = prefix[p.groups.G] * tiles_n;

  if (warp >= kEpilogueWarps) {
    registers_down<kOtherRegisters>();
    if (warp == kEpilogueWarps) {
      uint32_t it = 0, st = 0, phase = 0;  // stage and its round
      bool ok = true;
      for (unsigned t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile c = tile_at(p.groups, prefix, tiles_n, t);
        const int block0 = kSwiglu ? c.n : 2 * c.n, block1 = kSwiglu ? c.n + (F >> 7) : 2 * c.n + 1;
        const int halves = block1 < blocks_n ? 2 : 1;
        const unsigned char* scales = p.w_scales + (static_cast<long long>(c.group) * blocks_n + block0) * blocks_k * kScaleBytes;
        const long long second = static_cast<long long>(block1 - block0) * blocks_k * kScaleBytes;
        for (int kb = 0; kb < blocks_k; ++kb, ++it) {
          if (it >= num_stages) {
            ok = __all_sync(kFullMask, wait_or_quit(&s.empty[st], phase ^ 1, quit, err));
            if (!ok) break;
          }
          if (elect_one()) {
            unsigned char* a = stages + st * stage_bytes;
            unsigned char* f = a + 2 * kHalfBytes;
            unsigned char* b = a + kTokens;
            mbar_arrive_expect_tx(&s.full[st], halves * (kHalfLoad + kScaleBytes) + c.columns * kBlockK);
            tma_load_3d(a, &map_w, kb * kBlockK, block0 * 128, c.group, &s.full[st]);
            if (halves == 2) tma_load_3d(a + kHalfBytes, &map_w, kb * kBlockK, block1 * 128, c.group, &s.full[st]);
            bulk_load(f, scales + static_cast<long long>(kb) * kScaleBytes, kScaleBytes, &s.full[st]);
            if (halves == 2)
              bulk_load(f + kScaleBytes, scales + second + static_cast<long long>(kb) * kScaleBytes, kScaleBytes, &s.full[st]);
            for (int q = 0; q < c.columns; q += 16)
              tma_load_2d(b + q * kBlockK, &map_x, kb * kBlockK, static_cast<int>(c.row) + q, &s.full[st]);
          }
          __syncwarp();
          if (++st == num_stages) st = 0, phase ^= 1;
        }
      }
      // no load may outlive the block: wait for the last fill of every stage
      for (uint32_t i = it < num_stages ? 0 : it - num_stages; i < it; ++i) {
        int none = 0;
        wait_or_quit(&s.full[i % num_stages], (i / num_stages) & 1, &none, err);
      }
    } else if (warp <= kEpilogueWarps + 2) {
      const uint32_t odd = warp - kEpilogueWarps - 1;  // the warp issues the even or the odd blocks of k
      const uint64_t first = smem_desc(smem_u32(stages), 16, 1024);
      const uint64_t first_scales = scale_desc(smem_u32(stages) + 2 * kHalfBytes);
      const uint32_t a_scales = tmem + kWeightScales + odd * 8, b_scales = tmem + kTokenScales;
      uint32_t it = 0, st = 0, phase = 0, last = 0, last_phase = 0;
      bool used = false;
      bool ok = true;
      for (unsigned t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile c = tile_at(p.groups, prefix, tiles_n, t);
        const int halves = kSwiglu || 2 * c.n + 1 < blocks_n ? 2 : 1;
        const uint32_t desc = mma_mx_desc(128, c.columns, 0);
        for (int kb = 0; kb < blocks_k; ++kb, ++it) {
          const uint32_t at = st, round = phase;
          if (++st == num_stages) st = 0, phase ^= 1;
          if ((it & 1) != odd) continue;
          const uint32_t ac = it & (num_acc - 1), turn = (it / num_acc) & 1;
          ok = __all_sync(kFullMask, (it < num_acc || wait_or_quit(&s.acc_empty[ac], turn ^ 1, quit, err)) &&
                                         wait_or_quit(&s.full[at], round, quit, err));
          if (!ok) break;
          tmem_fence_after();
          if (elect_one()) {
            // descriptors count 16-byte units; 32 channels are two
            const uint64_t a = first + at * (stage_bytes >> 4), b = a + (kTokens >> 4);
            const uint64_t f = first_scales + at * (stage_bytes >> 4);
            const uint32_t d = tmem + ac * 2 * widest;
            for (int h = 0; h < halves; ++h) {
              tmem_copy_scales(a_scales + 4 * h, f + h * (kScaleBytes >> 4));
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_mx(d + h * widest, a + h * (kHalfBytes >> 4) + 2 * j, b + 2 * j,
                       desc | (static_cast<uint32_t>(j) << 4) | (static_cast<uint32_t>(j) << 29), a_scales + 4 * h,
                       b_scales, j > 0);
            }
            mma_commit(&s.acc_full[ac]);
            mma_commit(&s.empty[at]);
          }
          __syncwarp();
          used = true;
          last = ac;
          last_phase = turn;
        }
      }
      // nor may an MMA: its last accumulator is complete before TMEM goes back
      if (used) {
        int none = 0;
        wait_or_quit(&s.acc_full[last], last_phase, &none, err);
      }
    } else {
      // the tokens' scales of every block of k, with its operands
      uint32_t it = 0, st = 0, phase = 0;
      bool ok = true;
      for (unsigned t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile c = tile_at(p.groups, prefix, tiles_n, t);
        const float* sx = p.x.scales + (c.row + lane) * p.x.row_stride;
        const long long step = 32 * p.x.row_stride;
        for (int kb = 0; kb < blocks_k; ++kb, ++it) {
          if (it >= num_stages) {
            ok = __all_sync(kFullMask, wait_or_quit(&s.empty[st], phase ^ 1, quit, err));
            if (!ok) break;
          }
          const uint32_t dst = smem_u32(&s.x_scale[it % kScaleSlots][lane]);
#pragma unroll
          for (int j = 0; j < (kTileT + 31) / 32; ++j)
            if (32 * j + lane < c.rows) copy_async4(dst + j * 128, sx + j * step, true);
          copy_async_arrive(&s.full[st]);
          sx += p.x.group_stride;
          if (++st == num_stages) st = 0, phase ^= 1;
        }
      }
      asm volatile("cp.async.wait_all;" : : : "memory");
    }
  } else {
    registers_up<kEpilogueRegisters>();
    const int half = warp >> 2, quarter = warp & 3;
    const int in_half = quarter * 32 + lane;  // the thread's weight row in its half
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t it = 0;
    int turn = 0;
    bool ok = true;
    for (unsigned t = blockIdx.x; ok && t < tiles; t += gridDim.x, turn ^= 1) {
      const Tile c = tile_at(p.groups, prefix, tiles_n, t);
      const int chunks = c.columns >> 4;
      // a warp's columns: all of its half's, or half of both halves' (SwiGLU: 8
      // tokens' gates, then their up projections)
      const int first = kSwiglu ? half * (c.columns >> 1) : 0;
      float acc[kTileT];
#pragma unroll
      for (int j = 0; j < kTileT; ++j) acc[j] = 0.0f;
      for (int kb = 0; kb < blocks_k; ++kb, ++it) {
        const uint32_t ac = it & (num_acc - 1);
        ok = __all_sync(kFullMask, wait_or_quit(&s.acc_full[ac], (it / num_acc) & 1, quit, err));
        if (!ok) break;
        tmem_fence_after();
        const uint32_t d = lanes + ac * 2 * widest + (kSwiglu ? first : half * widest);
        const float* fx = s.x_scale[it % kScaleSlots] + first;  // of a row past the group's end: anything
        // 64 columns are on their way at a time; the accumulator goes back as soon as
        // the last are here
        uint32_t v[4][16];
        auto load = [&](int q) {
          if (q >= chunks) return;
          if constexpr (kSwiglu) {
            tmem_load8(d + 8 * q, v[q & 3]);
            tmem_load8(d + widest + 8 * q, v[q & 3] + 8);
          } else {
            tmem_load16(d + 16 * q, v[q & 3]);
          }
        };
        auto release = [&]() {
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.acc_empty[ac]);
        };
        auto add = [&](int q) {
          if (q >= chunks) return;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float f = fx[kSwiglu ? 8 * q + (j & 7) : 16 * q + j];
            acc[16 * q + j] = fmaf(__uint_as_float(v[q & 3][j]), f, acc[16 * q + j]);
          }
        };
#pragma unroll
        for (int q = 0; q < 4; ++q) load(q);
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_load_wait16(v[q]);
        if (chunks <= 4) {
          release();
#pragma unroll
          for (int q = 0; q < 4; ++q) add(q);
        } else {
#pragma unroll
          for (int q = 0; q < 3; ++q) add(q), load(q + 4);
          add(3);
#pragma unroll
          for (int q = 4; q < kChunks; ++q) tmem_load_wait16(v[q & 3]);
          release();
#pragma unroll
          for (int q = 4; q < kChunks; ++q) add(q);
        }
      }
      if (!ok) break;
      if constexpr (!kSwiglu) {
        const int n = c.n * 256 + half * 128 + in_half;
        uint16_t* o = p.out + c.row * p.N + n;
        if (n < p.N) {
#pragma unroll
          for (int j = 0; j < kTileT; ++j)
            if (j < c.rows) o[static_cast<long long>(j) * p.N] = static_cast<uint16_t>(pack_bf16x2(acc[j], 0.0f));
        }
      } else {
        const int mine = max(0, min(c.columns >> 1, c.rows - first));  // live tokens of this warp
        const long long row = c.row + first;
        float (*amax)[kTileT / 2] = s.amax[turn][half];
        float w[2] = {1.0f, 1.0f};
        if (p.row_weights) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (32 * i + lane < mine) w[i] = p.row_weights[row + 32 * i + lane];
        }
#pragma unroll
        for (int j = 0; j < kTileT / 2; ++j) {
          if (j < mine) {
            const float g = acc[16 * (j >> 3) + (j & 7)], u = acc[16 * (j >> 3) + 8 + (j & 7)];
            const float a = __fdividef(g, 1.0f + __expf(-g)) * u * __shfl_sync(kFullMask, w[j >> 5], j & 31);
            acc[16 * (j >> 3) + (j & 7)] = a;
            // a NaN does not enter the maximum
            const unsigned most = __reduce_max_sync(kFullMask, __float_as_uint(fmaxf(fabsf(a), 0.0f)));
            if (lane == 0) amax[quarter][j] = __uint_as_float(most);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.amax_full[half]);
        ok = __all_sync(kFullMask, wait_or_quit(&s.amax_full[half], turn, quit, err));
        if (!ok) break;
        unsigned char* o = p.act.data + row * F + c.n * 128 + in_half;
#pragma unroll
        for (int j = 0; j < kTileT / 2; ++j) {
          if (j < mine) {
            float inv;
            const float sc = group_scale(fmaxf(fmaxf(amax[0][j], amax[1][j]), fmaxf(amax[2][j], amax[3][j])), &inv);
            if (quarter == 0 && lane == (j & 31)) *p.act.scale(row + j, c.n) = sc;
            o[static_cast<long long>(j) * F] = static_cast<unsigned char>(pack_e4m3x2(acc[16 * (j >> 3) + (j & 7)] * inv, 0.0f));
          }
        }
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == kEpilogueWarps + 1) {
    tmem_fence_after();
    tmem_free(tmem, kTmemColumns);
  }
}

cudaError_t launch_grouped_matmul_w4(const Matmul4Args& p, int sms, cudaStream_t stream) {
  CUtensorMap map_x, map_w;
  cudaError_t e = make_byte_map(&map_x, p.x.data, p.K, p.groups.rows, 0, 16);
  if (e == cudaSuccess) e = make_e2m1_map(&map_w, p.w, p.K, p.N, p.groups.G, 128);
  if (e != cudaSuccess) return e;
  const bool swiglu = p.act.data != nullptr;
  int device = 0, smem = 0;  // all of it: the kernel decides on the stages
  if ((e = cudaGetDevice(&device)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, device)) != cudaSuccess)
    return e;
  const size_t least = sizeof(Shared) + sizeof(unsigned) * (p.groups.G + 1) + 1023 + 2 * (kTokens + kTileT * kBlockK);
  if (least > static_cast<size_t>(smem)) return cudaErrorInvalidValue;
  auto kernel = swiglu ? k_grouped_matmul_w4<true> : k_grouped_matmul_w4<false>;
  static std::atomic<unsigned long long> ready[2];  // devices set up, a bit each
  if ((e = set_up_kernel(reinterpret_cast<const void*>(kernel), ready[swiglu], kLaunchRegisters)) != cudaSuccess) return e;
  return launch_early(kernel, 1, dim3(sms), dim3(kThreads), smem, stream, map_x, map_w, p,
                      static_cast<uint32_t>(smem));
}

}  // namespace ep
