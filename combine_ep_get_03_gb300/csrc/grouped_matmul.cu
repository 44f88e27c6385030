// The experts' product on e4m3 rows: for a row r of group e
//   y[r, n] = sum_kb sx[r, kb] sw[e, n / 128, kb] sum_{k in block kb} x[r, k] w[e, n, k]
// with a scale for every 128 channels of a row and for every 128 x 128 block
// of the weights.  Stored as bf16, or (SwiGLU) taken through
//   a = row_weight silu(gate) up
// and stored as e4m3 with scales, the pre-activations kept as e4m3 if asked.
//
// Tile 128 rows x 256 columns, a block per SM that walks over tiles.  One
// warp loads 48 KB stages by TMA (128 channels of both operands, 128-byte
// swizzle); four MMAs a stage go into a fresh TMEM accumulator, since every
// 128 channels carry their own scale.  Two accumulators of 256 columns
// alternate, so while the tensor cores fill one, eight warps read the other (a
// thread owns a row, so its factor sx * sw is one number) and add it, scaled,
// to fp32 registers: 128 a thread.  The scales come with their operands: a
// fourth warp copies a block's 130 numbers to shared memory, asynchronously,
// so that the adding warps neither hold pointers nor wait for memory.  Each
// accumulator has its own issuing warp: a wait on a barrier that is already
// complete takes some 180 cycles here, two of them and the issue 620, more than
// the 512 of a stage's MMAs.
//
// Many rows: a stage's 48 KB are written to shared memory once and read once,
// some 750 cycles where the MMAs take 512 (without the loads the same kernel
// does 3.3 PFLOP/s, without the sums 2.2; a library product of 8 192^3 with one
// scale does 3.9); 32 768 rows, 7 168 -> 4 096: 897-923 us, 2.1 PFLOP/s, the tensor
// pipe 53 % active.  Few rows: the weights' stream; 32 experts of 2 048 -> 7 168 for
// 1 024 rows 77 us, 6.3 TB/s, and one token's eight experts of 7 168 -> 4 096
// 43 us, 5.4 TB/s (128 tiles on 152 SMs).  Pairs of blocks on a 256 x 256 tile
// halve the columns' traffic but lengthen the accumulators' round trip: decode
// 80 -> 113 us, prefill 900 -> 933 us, so blocks work alone.
//
// SwiGLU takes its 256 columns as gate 64, up 64, gate 64, up 64 so that a
// thread holds gate and up of the same channel and the row's 128-channel
// maximum needs one exchange between two threads.
#include <cuda.h>

#include <atomic>

#include "ep_internal.h"
#include "experts.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

constexpr int kTileM = 128, kTileN = 256, kBlockK = 128;
constexpr int kStages = 4;
constexpr int kRowBox = 32;  // rows a load brings
constexpr int kStageBytes = (kTileM + kTileN) * kBlockK;
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = (kEpilogueWarps + 4) * 32;  // a load, two MMA and a scale warp are the third warpgroup
// Registers: launched with 168 a thread; the third warpgroup hands most of its
// own to the two that hold accumulators.
constexpr int kLaunchRegisters = 168, kEpilogueRegisters = 232, kOtherRegisters = 40;
static_assert(kEpilogueWarps * 32 * kEpilogueRegisters + 4 * 32 * kOtherRegisters <= kThreads * kLaunchRegisters, "");
constexpr uint32_t kTmemColumns = 512;
constexpr int kScaleSlots = 8;  // blocks of k whose scales are kept: a slot's reader is done two accumulators earlier

struct Shared {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], amax_full;
  uint32_t tmem;
  int quit;
  unsigned sums[32];
  float x_scale[kScaleSlots][kTileM], w_scale[kScaleSlots][2];
  float amax[2][2][3][kTileM];  // [tile parity][half][gate, up, act][row]
};

struct Tile {
  int group, n;     // group and column tile
  long long row;    // first row
  int rows;         // live rows of the tile
};

__device__ __forceinline__ Tile tile_at(const GroupArgs& a, const unsigned* prefix, int tiles_n, unsigned t) {
  // tiles of a group are ordered column tile by column tile, row tiles inside
  const int g = find_group(prefix, a.G, t / static_cast<unsigned>(tiles_n));
  Tile r;
  long long start;
  const int count = group_span(a, g, &start, false);
  const int tiles_m = (count + kTileM - 1) / kTileM;
  const unsigned local = t - prefix[g] * tiles_n;
  r.group = g;
  r.n = tiles_m ? static_cast<int>(local / static_cast<unsigned>(tiles_m)) : 0;
  const int m = static_cast<int>(local) - r.n * tiles_m;
  r.row = start + static_cast<long long>(m) * kTileM;
  r.rows = tiles_m ? min(kTileM, count - m * kTileM) : 0;
  return r;
}

}  // namespace

template <bool kSwiglu>
__global__ void __launch_bounds__(kThreads, 1)
    k_grouped_matmul(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const MatmulArgs p) {
  extern __shared__ unsigned char raw[];
  unsigned char* stages = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Shared& s = *reinterpret_cast<Shared*>(stages + kStages * kStageBytes);
  unsigned* prefix = reinterpret_cast<unsigned*>(&s + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* quit = &s.quit;
  int* err = p.groups.err;

  if (threadIdx.x == 0) {
    // the loading thread's arrival and one of each of the scale warp's lanes
    for (int i = 0; i < kStages; ++i) mbar_init(&s.full[i], 1 + 32), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], kEpilogueWarps);
    mbar_init(&s.amax_full, kEpilogueWarps);
    s.quit = 0;
    mbar_init_fence();
    prefetch_map(&map_x);
    prefetch_map(&map_w);
  }
  if (warp == kEpilogueWarps + 1) tmem_alloc(&s.tmem, kTmemColumns);
  after_previous();
  groups_prefix(p.groups, kTileM, prefix, s.sums);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem;

  const int F = p.N >> 1;
  const int tiles_n = kSwiglu ? (F + kTileN / 2 - 1) / (kTileN / 2) : (p.N + kTileN - 1) / kTileN;
  const int blocks_k = p.K / kBlockK;
  const unsigned tiles = prefix[p.groups.G] * tiles_n;

  if (warp >= kEpilogueWarps) {
    registers_down<kOtherRegisters>();
    if (warp == kEpilogueWarps) {
      uint32_t it = 0;
      bool ok = true;
      for (unsigned t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile c = tile_at(p.groups, prefix, tiles_n, t);
        const int row_boxes = (c.rows + kRowBox - 1) / kRowBox;
        for (int kb = 0; kb < blocks_k; ++kb, ++it) {
          const int st = it % kStages;
          if (it >= kStages) {
            ok = __all_sync(kFullMask, wait_or_quit(&s.empty[st], ((it / kStages) & 1) ^ 1, quit, err));
            if (!ok) break;
          }
          if (elect_one()) {
            unsigned char* a = stages + st * kStageBytes;
            unsigned char* b = a + kTileM * kBlockK;
            // only the rows that are live, 32 at a time: the accumulators of the others
            // hold anything and are not stored
            mbar_arrive_expect_tx(&s.full[st], kTileN * kBlockK + row_boxes * kRowBox * kBlockK);
            for (int q = 0; q < row_boxes; ++q)
              tma_load_2d(a + q * kRowBox * kBlockK, &map_x, kb * kBlockK, static_cast<int>(c.row) + q * kRowBox, &s.full[st]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int n = kSwiglu ? c.n * 128 + (q >> 1) * 64 + (q & 1) * F : c.n * kTileN + q * 64;
              tma_load_3d(b + q * 64 * kBlockK, &map_w, kb * kBlockK, n, c.group, &s.full[st]);
            }
          }
          __syncwarp();
        }
      }
      // no load may outlive the block: wait for the last fill of every stage
      for (uint32_t i = it < kStages ? 0 : it - kStages; i < it; ++i) {
        int none = 0;
        wait_or_quit(&s.full[i % kStages], (i / kStages) & 1, &none, err);
      }
    } else if (warp <= kEpilogueWarps + 2) {
      const int ac = warp - kEpilogueWarps - 1;  // the warp's accumulator: even or odd blocks of k
      constexpr uint32_t desc = mma_desc(kTileM, kTileN, false);
      const uint64_t first = smem_desc(smem_u32(stages), 16, 1024);
      const unsigned mine = tiles > blockIdx.x ? (tiles - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
      const uint32_t all = mine * blocks_k;  // blocks of k of this block's tiles
      uint32_t it = ac;
      for (; it < all; it += 2) {
        const int st = it % kStages;
        const bool ok = __all_sync(kFullMask, (it < 2 || wait_or_quit(&s.acc_empty[ac], ((it >> 1) & 1) ^ 1, quit, err)) &&
                                                  wait_or_quit(&s.full[st], (it / kStages) & 1, quit, err));
        if (!ok) break;
        tmem_fence_after();
        if (elect_one()) {
          // descriptors count 16-byte units; 32 channels are two
          const uint64_t a = first + st * (kStageBytes >> 4), b = a + (kTileM * kBlockK >> 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_f8(tmem + ac * kTileN, a + 2 * j, b + 2 * j, desc, j > 0);
          mma_commit(&s.acc_full[ac]);
          mma_commit(&s.empty[st]);
        }
        __syncwarp();
      }
      // nor may an MMA: its last accumulator is complete before TMEM goes back
      if (it >= 2) {
        int none = 0;
        wait_or_quit(&s.acc_full[ac], ((it - 2) >> 1) & 1, &none, err);
      }
    } else {
      // the scales of every block of k, with its operands: 128 rows' and the
      // weights' two (the tile's halves, or gate and up)
      const int Gn = (p.N + 127) >> 7;
      uint32_t it = 0;
      bool ok = true;
      for (unsigned t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile c = tile_at(p.groups, prefix, tiles_n, t);
        const float* sx = p.x.scales + (c.row + lane) * p.x.row_stride;
        const long long step = 32 * p.x.row_stride;
        const int n0 = kSwiglu ? c.n + (lane & 1) * (F >> 7) : c.n * 2 + (lane & 1);
        const float* sw = p.w_scales + (static_cast<long long>(c.group) * Gn + min(n0, Gn - 1)) * blocks_k;
        for (int kb = 0; kb < blocks_k; ++kb, ++it) {
          const int st = it % kStages, slot = it % kScaleSlots;
          if (it >= kStages) {
            ok = __all_sync(kFullMask, wait_or_quit(&s.empty[st], ((it / kStages) & 1) ^ 1, quit, err));
            if (!ok) break;
          }
          const uint32_t dst = smem_u32(&s.x_scale[slot][lane]);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (32 * j + lane < c.rows) copy_async4(dst + j * 128, sx + j * step, true);
          if (lane < 2) copy_async4(smem_u32(&s.w_scale[slot][lane]), sw + kb, true);
          copy_async_arrive(&s.full[st]);
          sx += p.x.group_stride;
        }
      }
      asm volatile("cp.async.wait_all;" : : : "memory");
    }
  } else {
    registers_up<kEpilogueRegisters>();
    const int half = warp >> 2, quarter = warp & 3;
    const int in_tile = quarter * 32 + lane;  // the thread's row in the tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * (kTileN / 2);
    const bool wide = kSwiglu ? false : ((reinterpret_cast<uintptr_t>(p.out) | (static_cast<uintptr_t>(p.N) * 2)) & 31) == 0;
    uint32_t it = 0;
    int turn = 0;
    bool ok = true;
    for (unsigned t = blockIdx.x; ok && t < tiles; t += gridDim.x, turn ^= 1) {
      const Tile c = tile_at(p.groups, prefix, tiles_n, t);
      const long long row = c.row + in_tile;
      const bool live = in_tile < c.rows;
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
      for (int kb = 0; kb < blocks_k; ++kb, ++it) {
        const int ac = it & 1;
        ok = __all_sync(kFullMask, wait_or_quit(&s.acc_full[ac], (it >> 1) & 1, quit, err));
        if (!ok) break;
        tmem_fence_after();
        // 32 columns are on their way while the 32 before them are added
        uint32_t v[2][32];
        tmem_load32(lanes + ac * kTileN, v[0]);
        const int slot = it % kScaleSlots;
        const float fx = s.x_scale[slot][in_tile];  // of a row past the group's end: anything
        const float f0 = fx * s.w_scale[slot][kSwiglu ? 0 : half], f1 = kSwiglu ? fx * s.w_scale[slot][1] : f0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_load_wait(v[q & 1]);
          if (q < 3) {
            tmem_load32(lanes + ac * kTileN + (q + 1) * 32, v[(q + 1) & 1]);
          } else {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.acc_empty[ac]);
          }
          const float f = kSwiglu && q >= 2 ? f1 : f0;
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[q * 32 + j] = fmaf(__uint_as_float(v[q & 1][j]), f, acc[q * 32 + j]);
        }
      }
      if (!ok) break;
      if constexpr (!kSwiglu) {
        const int col = c.n * kTileN + half * 128;
        if (live) {
          uint16_t* o = p.out + row * p.N + col;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = pack_bf16x2(acc[q * 16 + 2 * j], acc[q * 16 + 2 * j + 1]);
            if (col + q * 16 + 16 <= p.N)
              store32(o + q * 16, v, wide);
            else if (col + q * 16 + 8 <= p.N)
              *reinterpret_cast<uint4*>(o + q * 16) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      } else {
        const int f = c.n * 128 + half * 64;
        const float w = live && p.row_weights ? p.row_weights[row] : 1.0f;
        const bool keep = p.pre.data != nullptr;
        float (*amax)[3][kTileM] = s.amax[turn];
        float ag = 0.0f, au = 0.0f, aa = 0.0f;
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          const float g = acc[j], u = acc[64 + j];
          ag = fmaxf(ag, fabsf(g));
          au = fmaxf(au, fabsf(u));
          aa = fmaxf(aa, fabsf(__fdividef(g, 1.0f + __expf(-g)) * u * w));
        }
        amax[half][0][in_tile] = ag;
        amax[half][1][in_tile] = au;
        amax[half][2][in_tile] = aa;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.amax_full);
        ok = __all_sync(kFullMask, wait_or_quit(&s.amax_full, turn, quit, err));
        if (!ok) break;
        if (live) {
          float inv;
          uint32_t q[16];
          if (keep) {
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              const float sc = group_scale(fmaxf(amax[0][part][in_tile], amax[1][part][in_tile]), &inv);
              if (half == 0) *p.pre.scale(row, c.n + part * (F >> 7)) = sc;
#pragma unroll
              for (int j = 0; j < 16; ++j) q[j] = quant4(acc + part * 64 + 4 * j, inv);
              unsigned char* o = p.pre.data + row * p.N + part * F + f;
              const bool w32 = (reinterpret_cast<uintptr_t>(o) & 31) == 0;
              store32(o, q, w32);
              store32(o + 32, q + 8, w32);
            }
          }
          const float sc = group_scale(fmaxf(amax[0][2][in_tile], amax[1][2][in_tile]), &inv);
          if (half == 0) *p.act.scale(row, c.n) = sc;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              a[i] = __fdividef(acc[4 * j + i], 1.0f + __expf(-acc[4 * j + i])) * acc[64 + 4 * j + i] * w;
            q[j] = quant4(a, inv);
          }
          unsigned char* o = p.act.data + row * F + f;
          const bool w32 = (reinterpret_cast<uintptr_t>(o) & 31) == 0;
          store32(o, q, w32);
          store32(o + 32, q + 8, w32);
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

namespace {

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encode_tiled() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

}  // namespace

namespace {

cudaError_t make_map(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base, int width, long long rows,
                     int planes, int box_rows) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t rank = planes > 0 ? 3 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(planes > 0 ? planes : 1)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(width) * size, static_cast<cuuint64_t>(width) * size * rows};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return enc(map, type, rank, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t make_byte_map(CUtensorMap* map, const void* base, int width, long long rows, int planes, int box_rows) {
  return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, width, rows, planes, box_rows);
}
cudaError_t make_tensor_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
                            const cuuint64_t* strides, const cuuint32_t* box, bool swizzle) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  return enc(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}
cudaError_t make_bf16_map(CUtensorMap* map, const void* base, int width, long long rows, int box_rows) {
  return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, width, rows, 0, box_rows);
}

cudaError_t launch_grouped_matmul(const MatmulArgs& p, int sms, cudaStream_t stream) {
  CUtensorMap map_x, map_w;
  cudaError_t e = make_byte_map(&map_x, p.x.data, p.K, p.groups.rows, 0, kRowBox);
  if (e == cudaSuccess) e = make_byte_map(&map_w, p.w, p.K, p.N, p.groups.G, 64);
  if (e != cudaSuccess) return e;
  const bool swiglu = p.act.data != nullptr;
  const size_t smem = 1024 + static_cast<size_t>(kStages) * kStageBytes + sizeof(Shared) + sizeof(unsigned) * (p.groups.G + 1);
  auto kernel = swiglu ? k_grouped_matmul<true> : k_grouped_matmul<false>;
  static std::atomic<unsigned long long> ready[2];  // devices set up, a bit each
  if ((e = set_up_kernel(reinterpret_cast<const void*>(kernel), ready[swiglu], kLaunchRegisters)) != cudaSuccess) return e;
  return launch_early(kernel, 1, dim3(sms), dim3(kThreads), smem, stream, map_x, map_w, p);
}

}  // namespace ep
