// Weight gradient of the experts' product from 8-bit rows:
//   dw[e, n, k] = sum over the rows r of group e of dy[r, n] x[r, k],
// both e4m3 with a scale for every 128 channels of a row.
//
// The contraction runs over rows, and both scales change with the row, so they
// cannot be taken out of the sum: the operands are multiplied by their scales
// in fp32 on the way to shared memory, rounded once to f16, and go through f16
// tensor-core instructions with fp32 accumulation.  The scales of an operand's
// 128 channels are first divided by the power of two that brings the largest
// of the group's rows to [64, 128) (448 x 128 still fits f16), which is put
// back on the sums.  So a term is off by 2^-10 of itself, a quarter of the bf16
// result's own 2^-8, as long as both values are 2^-28 of their channels' largest
// possible (448 times that scale) or more; f16's subnormal step is 2^-39 of it.
// bf16 operands would keep any range but round to 2^-8 each.  Scale and product
// both rounded to f16 (no fp32 arithmetic) 386 us, this 409-414; a scale split
// in two f16 numbers 412, and with the range above 418.
//
// Shared memory is what bounds it: a widened 64-row stage is written once and
// read once per MMA.  So two blocks on neighbouring SMs share a tile of 256 (n)
// x 256 (k): each widens its 128 columns of dy and of x, 32 KB a stage instead
// of the 48 KB of a 128 x 256 tile of its own, for the same MMA time.  Two
// warps fetch e4m3 rows (TMA) and scales (asynchronous copies) four stages
// ahead, across tiles; four teams of four warps take a stage each in turn,
// widen it and store it with the 128-byte swizzle, rows along the long axis
// (both operands "MN major", so nothing is transposed).  One warp of the first
// block issues four MMAs a stage; four warps send the previous tile from the
// other TMEM accumulator out through shared memory; one looks up the next
// tiles' largest scales.  Rows past the group's end enter as zeros.
//
// 16 experts, 16 384 rows, 2 048 x 7 168: 409-414 us, 1.17 PFLOP/s; 61 % of the
// issue slots are taken, the load-store pipe is busy 52 % of the cycles and the
// tensor cores' operand reads take about another quarter of the same memory.
// Measured with two f16 roundings (386 us): one block alone on 128 x 256 614 us;
// rows by plain loads instead of TMA 464 us at best; 32-byte stores of the result
// straight from registers 410 us.
#include "ep_internal.h"
#include "experts.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

constexpr int kPair = 256;     // the pair's tile: 256 x 256
constexpr int kOwn = 128;      // a block's columns of dy, of x and rows of the accumulator
constexpr int kRows = 64;
constexpr int kStages = 4;     // widened
constexpr int kRawStages = 4;  // as fetched; both a multiple of the teams: a stage belongs to one
constexpr int kChunkBytes = kRows * 128;  // 64 columns of f16
constexpr int kStageBytes = 2 * kOwn / 64 * kChunkBytes;
constexpr int kRawBytes = 2 * kOwn * kRows, kScaleBytes = 2 * 4 * kRows;  // dy, x; their scales
constexpr int kOutBytes = 32 * 128;  // 32 rows of 64 bf16
constexpr int kTeams = 4, kTeamWarps = 4, kPass = 4 * kTeamWarps, kLoadWarps = kTeams * kTeamWarps, kStoreWarps = 4;
constexpr int kMmaWarp = kLoadWarps + kStoreWarps, kScaleWarp = kMmaWarp + 1, kFetchWarp = kMmaWarp + 2;
constexpr int kFetchWarps = 2;
constexpr int kThreads = (kFetchWarp + kFetchWarps) * 32;
constexpr uint32_t kTmemColumns = 512;
constexpr int kExponents = 8;  // tiles whose exponents are kept: at least stages + 2

struct Shared {
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], exp_full[kExponents], exp_empty[kExponents];
  uint32_t tmem;
  int quit;
  int exponent[kExponents][3];  // of the block's dy, of both halves of x
};
// Shared memory without the groups' counts, which follow it: 4096 of them fit.
constexpr size_t kSharedBytes = static_cast<size_t>(kStages) * kStageBytes + kRawStages * (kRawBytes + kScaleBytes) +
                                kStoreWarps * kOutBytes + sizeof(Shared);
static_assert(kSharedBytes + sizeof(int) * kMaxGroups <= 227 * 1024, "");

// The pair's tiles that have rows, one after another.
struct Walk {
  const GroupArgs* groups;
  const int* counts;  // rows of every group, in shared memory
  int tiles_n, tiles_k;
  unsigned t, tiles, step;
  int group, n, k, rows;
  __device__ __forceinline__ void set() {
    const unsigned row = t / static_cast<unsigned>(tiles_k);
    k = static_cast<int>(t - row * tiles_k);
    group = static_cast<int>(row / static_cast<unsigned>(tiles_n));
    n = static_cast<int>(row - group * tiles_n);
    rows = counts[group];
  }
  __device__ __forceinline__ bool settle() {  // at t or after it
    for (; t < tiles; t += step) {
      set();
      if (rows) return true;
    }
    return false;
  }
  __device__ __forceinline__ bool next() {
    t += step;
    return settle();
  }
  __device__ __forceinline__ int blocks() const { return (rows + kRows - 1) / kRows; }
  __device__ __forceinline__ long long row() const {
    return groups->offset ? static_cast<long long>(groups->offset[group]) : group * groups->rows_per_group;
  }
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

// Two products as f16, rounded once (the products in fp32, one instruction for both).
__device__ __forceinline__ uint32_t scaled_f16x2(float a, float b, float scale) {
  uint32_t r;
  asm("{\n .reg .b64 t, u;\n .reg .f32 x, y;\n mov.b64 t, {%1, %2};\n mov.b64 u, {%3, %3};\n mul.rn.f32x2 t, t, u;\n"
      " mov.b64 {x, y}, t;\n cvt.rn.f16x2.f32 %0, y, x;\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(scale));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" : : "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 codes times their scale, as f16 at the two shared-memory addresses of
// their 16-byte units.
__device__ __forceinline__ void store_chunk(uint32_t lo, uint32_t hi, const uint4& q, float scale) {
  uint32_t h[8];
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    e4m3x4_to_f32(w[i], f);
    h[2 * i] = scaled_f16x2(f[0], f[1], scale);
    h[2 * i + 1] = scaled_f16x2(f[2], f[3], scale);
  }
  sts128(lo, h[0], h[1], h[2], h[3]);
  sts128(hi, h[4], h[5], h[6], h[7]);
}

// 2^e that brings m to [64, 128) (towards it, where m is subnormal); a largest
// scale of 0 leaves the scales as they are.
__device__ __forceinline__ int exponent_of(float m) { return m > 0.0f ? max(-126, ilogbf(m) - 6) : 0; }
__device__ __forceinline__ float finite_size(float scale) {
  const float m = fabsf(scale);
  return m <= 3.402823466e38f ? m : 0.0f;
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1) 
    k_weight_grad(const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_dw,
                  const __grid_constant__ WeightGradArgs p) {
  extern __shared__ __align__(1024) unsigned char stages[];
  unsigned char* raws = stages + kStages * kStageBytes;
  unsigned char* outs = raws + kRawStages * kRawBytes;  // what the storing warps have on its way out
  unsigned char* raw_scales = outs + kStoreWarps * kOutBytes;
  Shared& s = *reinterpret_cast<Shared*>(raw_scales + kRawStages * kScaleBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* quit = &s.quit;
  int* err = p.groups.err;
  const int rank = static_cast<int>(cluster_rank());
  int* counts = reinterpret_cast<int*>(&s + 1);
  if (threadIdx.x == 0) {
    // the fetching thread's own arrival and one of every lane's copies
    for (int i = 0; i < kRawStages; ++i) mbar_init(&s.raw_full[i], 1 + 32), mbar_init(&s.raw_empty[i], kTeamWarps);
    for (int i = 0; i < kStages; ++i) mbar_init(&s.full[i], 2 * kTeamWarps), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.acc_full[i], 1), mbar_init(&s.acc_empty[i], 2 * kStoreWarps);
    for (int i = 0; i < kExponents; ++i) mbar_init(&s.exp_full[i], 1), mbar_init(&s.exp_empty[i], kStoreWarps);
    s.quit = 0;
    mbar_init_fence();
  }
  if (warp == kMmaWarp) pair_tmem_alloc(&s.tmem, kTmemColumns);
  after_previous();
  for (int g = threadIdx.x; g < p.groups.G; g += kThreads) {
    long long start;
    counts[g] = group_span(p.groups, g, &start, blockIdx.x == 0);
  }
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = s.tmem;
  Walk w;
  w.groups = &p.groups;
  w.counts = counts;
  w.tiles_n = (p.N + kPair - 1) / kPair;
  w.tiles_k = (p.K + kPair - 1) / kPair;
  w.tiles = static_cast<unsigned>(p.groups.G) * w.tiles_n * w.tiles_k;
  w.t = blockIdx.x >> 1;
  w.step = gridDim.x >> 1;

  if (warp < kLoadWarps) {
    const int team = warp / kTeamWarps;
    // A warp's 32 chunks of 16 channels are eight of each of four rows.  Eight
    // lanes in a row hold four chunks of each of two rows r and r ^ 5.  Both
    // tiles are swizzled by the row (chunk or 16-byte unit ^ row mod 8): the raw
    // chunks of the two rows differ in bit 2, the widened units 2 (c mod 4) and
    // the next in bit 0, so a phase of either 16-byte access meets all banks once.
    const int pair = (warp % kTeamWarps) * 2 + (lane >> 4);
    const int my_row = (pair >> 2) * 8 + ((pair & 3) ^ ((lane & 4) ? 5 : 0));
    const int c4 = lane & 3, chunk = c4 + ((lane >> 3) & 1) * 4;
    const uint32_t line = smem_u32(stages) + (chunk >> 2) * kChunkBytes + my_row * 128;
    const uint32_t unit_lo = line + (((2 * c4) ^ (my_row & 7)) << 4);
    const uint32_t unit_hi = line + (((2 * c4 + 1) ^ (my_row & 7)) << 4);
    const unsigned char* my_raw = raws + my_row * kOwn + ((chunk ^ (my_row & 7)) << 4);
    const float* my_scales = reinterpret_cast<const float*>(raw_scales) + my_row;
    Cursor now;
    now.begin(w);
    for (int i = 0; i < team; ++i) now.step();
    uint32_t tile = ~0u;  // whose exponents `dy_down` and `x_down` hold
    float dy_down = 1.0f, x_down = 1.0f;
    for (uint32_t it = team; now.on; it += kTeams) {
      const int st = it % kStages, rs = it % kRawStages;
      bool ok = true;
      if (now.used != tile) {
        tile = now.used;
        const int e = tile % kExponents;
        ok = wait_or_quit(&s.exp_full[e], (tile / kExponents) & 1, quit, err);
        dy_down = power_of_two(-s.exponent[e][0]);
        x_down = power_of_two(-s.exponent[e][1 + rank]);
      }
      ok = ok && wait_or_quit(&s.raw_full[rs], (it / kRawStages) & 1, quit, err);
      if (!__all_sync(kFullMask, ok)) break;
      const unsigned char* raw_at = my_raw + rs * kRawBytes;
      const float* scales_at = my_scales + rs * (kScaleBytes / 4);
      const int left = now.w.rows - now.b * kRows - my_row;  // rows past it are another group's
      uint4 q[2][kRows / kPass];
      float f[2][kRows / kPass];
#pragma unroll
      for (int j = 0; j < kRows / kPass; ++j) {
        const bool on = j * kPass < left;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          q[h][j] = on ? lds128(raw_at + h * kOwn * kRows + j * kPass * kOwn) : make_uint4(0, 0, 0, 0);
          f[h][j] = scales_at[h * kRows + j * kPass] * (h ? x_down : dy_down);
        }
      }
      if (it >= kStages &&
          !__all_sync(kFullMask, wait_or_quit<true>(&s.empty[st], ((it / kStages) & 1) ^ 1, quit, err)))
        break;
      const uint32_t lo = unit_lo + st * kStageBytes, hi = unit_hi + st * kStageBytes;
#pragma unroll
      for (int j = 0; j < kRows / kPass; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          store_chunk(lo + h * 2 * kChunkBytes + j * kPass * 128, hi + h * 2 * kChunkBytes + j * kPass * 128, q[h][j], f[h][j]);
      fence_proxy_async_smem();
      __syncwarp();
      // the raw stage goes back only now: its loads are complete once their values
      // have been stored, not when they have been issued
      if (lane == 0) {
        mbar_arrive(&s.raw_empty[rs]);
        mbar_arrive_first(&s.full[st]);
      }
      for (int i = 0; i < kTeams; ++i) now.step();
    }
  } else if (warp >= kFetchWarp) {
    const int mine = warp - kFetchWarp;
    Cursor c;
    c.begin(w);
    for (int i = 0; i < mine; ++i) c.step();
    uint32_t it = mine;
    for (; c.on; it += kFetchWarps) {
      const int n = c.w.n * 2 + rank, k = c.w.k * 2 + rank;
      const bool in_n = n < (p.N >> 7), in_k = k < (p.K >> 7);
      const int rs = it % kRawStages;
      const long long r = c.w.row() + c.b * kRows;
      if (it >= kRawStages &&
          !__all_sync(kFullMask, wait_or_quit(&s.raw_empty[rs], ((it / kRawStages) & 1) ^ 1, quit, err)))
        break;
      if (elect_one()) {
        // columns past the matrix and rows past the buffer read as zeros
        mbar_arrive_expect_tx(&s.raw_full[rs], kRawBytes);
        tma_load_2d(raws + rs * kRawBytes, &map_dy, n * kOwn, static_cast<int>(r), &s.raw_full[rs]);
        tma_load_2d(raws + rs * kRawBytes + kOwn * kRows, &map_x, k * kOwn, static_cast<int>(r), &s.raw_full[rs]);
      }
      __syncwarp();
      const uint32_t dst = smem_u32(raw_scales + rs * kScaleBytes) + lane * 4;
      const float* dy_scale = p.dy.scale(r + lane, n);
      const float* x_scale = p.x.scale(r + lane, k);
      const int left = c.w.rows - c.b * kRows - lane;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool live = 32 * j < left;
        copy_async4(dst + j * 128, live && in_n ? dy_scale + j * 32 * p.dy.row_stride : p.dy.scales, live && in_n);
        copy_async4(dst + 4 * kRows + j * 128, live && in_k ? x_scale + j * 32 * p.x.row_stride : p.x.scales, live && in_k);
      }
      copy_async_arrive(&s.raw_full[rs]);
      for (int i = 0; i < kFetchWarps; ++i) c.step();
    }
    // no copy may outlive the block: wait for the last fill of every stage
    for (uint32_t i = it < kRawStages ? mine : it - kRawStages; i < it; i += kFetchWarps) {
      int none = 0;
      wait_or_quit(&s.raw_full[i % kRawStages], (i / kRawStages) & 1, &none, err);
    }
  } else if (warp == kScaleWarp) {
    // the exponents of the tiles to come
    uint32_t used = 0;
    for (bool on = w.settle(); on; on = w.next(), ++used) {
      const int e = used % kExponents;
      if (used >= kExponents &&
          !__all_sync(kFullMask, wait_or_quit(&s.exp_empty[e], ((used / kExponents) & 1) ^ 1, quit, err)))
        break;
      const int n = w.n * 2 + rank, k = w.k * 2;
      const bool in_n = n < (p.N >> 7), second = k + 1 < (p.K >> 7);
      const float* ys = p.dy.scale(w.row(), n);
      const float* xs = p.x.scale(w.row(), k);
      float m[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll 8
      for (int r = lane; r < w.rows; r += 32) {
        if (in_n) m[0] = fmaxf(m[0], finite_size(ys[r * p.dy.row_stride]));
        m[1] = fmaxf(m[1], finite_size(xs[r * p.x.row_stride]));
        if (second) m[2] = fmaxf(m[2], finite_size(xs[r * p.x.row_stride + p.x.group_stride]));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int h = 0; h < 3; ++h) m[h] = fmaxf(m[h], __shfl_xor_sync(kFullMask, m[h], d));
      if (lane == 0) {
#pragma unroll
        for (int h = 0; h < 3; ++h) s.exponent[e][h] = exponent_of(m[h]);
        mbar_arrive(&s.exp_full[e]);
      }
      __syncwarp();
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t desc = mma_desc(kPair, kPair, true);
    const uint64_t first = smem_desc(smem_u32(stages), kChunkBytes, 1024);
    uint32_t it = 0, used = 0;
    bool ok = true;
    for (bool on = rank == 0 && w.settle(); ok && on; on = w.next()) {
      const int ac = used & 1, blocks = w.blocks();
      ok = __all_sync(kFullMask, used < 2 || wait_or_quit<true>(&s.acc_empty[ac], ((used >> 1) & 1) ^ 1, quit, err));
      if (!ok) break;
      int left = w.rows;
      for (int b = 0; b < blocks; ++b, ++it, left -= kRows) {
        const int st = it % kStages;
        ok = __all_sync(kFullMask, wait_or_quit<true>(&s.full[st], (it / kStages) & 1, quit, err));
        if (!ok) break;
        tmem_fence_after();
        if (elect_one()) {
          // descriptors count 16-byte units; an MMA takes 16 rows of 128 bytes
          const uint64_t dy = first + st * (kStageBytes >> 4), x = dy + (2 * kChunkBytes >> 4);
#pragma unroll
          for (int j = 0; j < kRows / 16; ++j)
            if (16 * j < left) pair_mma_f16(tmem + ac * kPair, dy + 128 * j, x + 128 * j, desc, b > 0 || j > 0);
          pair_mma_commit(&s.empty[st]);
        }
        __syncwarp();
      }
      // also after a wait that gave up: what was issued ends before TMEM goes back
      if (elect_one()) pair_mma_commit(&s.acc_full[ac]);
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
    // 64 columns of the warp's 32 rows at a time go through shared memory, so
    // that they leave as whole lines: 32-byte stores into 32 rows cost the
    // load-store pipe, which bounds the widening, four times as much
    unsigned char* out = outs + quarter * kOutBytes;
    auto send = [&](const uint32_t* x, int column, int row) {
      if (lane == 0) bulk_wait_read<0>();  // the 64 columns before have left
      __syncwarp();
      const uint32_t line = smem_u32(out) + lane * 128;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        sts128(line + ((u ^ (lane & 7)) << 4), x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&map_dw, out, column, row);
        bulk_commit();
      }
    };
    uint32_t used = 0;
    for (; w.t < w.tiles; w.t += w.step) {
      w.set();
      const int n = w.n * kPair + rank * kOwn, k = w.k * kPair;
      const int columns = n < p.N ? min(kPair, p.K - k) : 0;
      const int row = w.group * p.N + n + quarter * 32;
      uint32_t x[32];
      if (w.rows == 0) {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = 0u;
        for (int q = 0; q < columns; q += 64) send(x, k + q, row);
        continue;
      }
      const int ac = used & 1, e = used % kExponents;
      if (!__all_sync(kFullMask, wait_or_quit(&s.exp_full[e], (used / kExponents) & 1, quit, err) &&
                                     wait_or_quit<true>(&s.acc_full[ac], (used >> 1) & 1, quit, err)))
        break;
      tmem_fence_after();
      // each half's 2^(dy's + x's exponent) as two factors: the sum may be beyond
      // what one fp32 number holds
      float up[2], rest[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int sum = s.exponent[e][0] + s.exponent[e][1 + h], first = max(-126, min(126, sum));
        up[h] = power_of_two(first);
        rest[h] = power_of_two(max(-126, min(126, sum - first)));
      }
#pragma unroll
      for (int q = 0; q < kPair / 64; ++q) {
        const float f = up[q >> 1], f2 = rest[q >> 1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
          tmem_load32(lanes + ac * kPair + q * 64 + h * 32, v);
          tmem_load_wait(v);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            x[h * 16 + j] = pack_bf16x2(__uint_as_float(v[2 * j]) * f * f2, __uint_as_float(v[2 * j + 1]) * f * f2);
        }
        if (q == kPair / 64 - 1) {
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_first(&s.acc_empty[ac]);
        }
        if (q * 64 < columns) send(x, k + q * 64, row);
      }
      // the exponents have been used, not only read
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.exp_empty[e]);
      ++used;
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  cluster_sync();  // the other block arrives on this one's barriers until here
  if (warp == kMmaWarp) {
    tmem_fence_after();
    pair_tmem_free(tmem, kTmemColumns);
  }
}

cudaError_t launch_weight_grad(const WeightGradArgs& p, int sms, cudaStream_t stream) {
  CUtensorMap map_dy, map_x, map_dw;
  cudaError_t e = make_byte_map(&map_dy, p.dy.data, p.N, p.groups.rows, 0, kRows);
  if (e == cudaSuccess) e = make_byte_map(&map_x, p.x.data, p.K, p.groups.rows, 0, kRows);
  if (e == cudaSuccess) e = make_bf16_map(&map_dw, p.dw, p.K, static_cast<long long>(p.groups.G) * p.N, 32);
  static std::atomic<unsigned long long> ready;  // devices set up, a bit each
  if (e == cudaSuccess) e = set_up_kernel(reinterpret_cast<const void*>(k_weight_grad), ready, 0);
  if (e != cudaSuccess) return e;
  const size_t smem = kSharedBytes + sizeof(int) * p.groups.G;
  // pairs of blocks: an even number of SMs, two at least
  return launch_early(k_weight_grad, 2, dim3(sms < 2 ? 2 : sms & ~1), dim3(kThreads), smem, stream, map_dy, map_x, map_dw, p);
}

}  // namespace ep
