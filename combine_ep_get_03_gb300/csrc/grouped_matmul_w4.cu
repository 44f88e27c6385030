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
// x's scales are arbitrary; the adding warps read it and add it to fp32 registers
// times its column's scale.
//
// Tile 256 weight rows (two halves of 128, in SwiGLU the gate's and the up
// projection's of the same channels) x up to 112 tokens; two accumulators of
// both halves take 448 TMEM columns, the scales 20 more.  With few tokens a
// tile an accumulator holds two or four blocks of k, as many as are handed over
// together, and the ring has more stages.  A block of k is always added alone and in
// order, so a row's bits do not depend on the other rows, the tile or the SMs.
//
// Few rows: the stream of weights.  128 tokens by 8 of 32 experts, 2 048 -> 7 168: 50 us
// (8-bit 77), 5.4 TB/s; one token's eight experts of 7 168 -> 4 096: 26 us (43), of which 5
// are start and end; with experts enough to fill the SMs four times 90 % of the copy
// rate.  The loads alone take 45 of the 50 us (39 at the copy rate): TMA's spreading costs
// some.  Many rows: the accumulators' round from the MMAs to the warps that add and back,
// some 1 150 cycles a stage; 16 384 rows, 7 168 -> 2 x 2 048: 560 to 587 us over several runs,
// 1.7 PFLOP/s, at 1.3 of 1.4 kW; plain, 2 048 -> 7 168: 349 us, 1.4 PFLOP/s (8-bit weights 278:
// they are the faster ones there).  Of a stage's cycles shared memory is busy for 850
// (weights and tokens are written once and read once, the tokens twice): without the
// sums SwiGLU's takes 375 us.
#include <cuda.h>

#include <atomic>

#include "ep_internal.h"
#include "experts.cuh"
#include "pairs.cuh"
#include "tcgen05.cuh"

namespace ep {

// Both halves' codes, their exponents; 16, 32 and 64 rows of tokens.
struct Matmul4Maps {
  CUtensorMap w, scales, x[3];
};

namespace {

constexpr int kTileT = kTile4Rows, kBlockK = 128;
constexpr int kChunks = kTileT / 16;
constexpr int kMaxStages = 8;
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
// TMEM: two accumulators, behind them eight columns of exponents for each of their
// blocks of k (an MMA's are its accumulator's, so nothing overwrites those of one
// that runs), the tokens' scales at the end.
constexpr uint32_t kTokenScales = kTmemColumns - 4;
static_assert(2 * (2 * kTileT + 8) <= kTokenScales && 2 * 2 * (2 * 48 + 8) <= kTokenScales && 2 * 4 * (2 * 16 + 8) <= kTokenScales, "");
// Blocks of k whose token scales are kept, and words for them.  A slot is filled
// again when the MMAs of `kept - stages` blocks later are done; the warps that
// add may then be reading those of three hand-overs before.
constexpr int kScaleWords = 1792;
static_assert(16 * kTileT <= kScaleWords && 32 * 48 <= kScaleWords, "");

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], amax_full[2], drained[2];
  uint32_t tmem;
  int quit, columns;
  unsigned sums[32];
  alignas(16) float x_scale[kScaleWords];
  alignas(16) float amax[2][2][kTileT / 2][4];  // [tile parity][half][token][warp]
  float inv[2][4][kTileT / 2];                  // [half][warp][token]
};

// The same value in every lane, said so that the compiler keeps it, and what is
// made of it, in uniform registers: MMAs and tensor loads take their operands there.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(kFullMask, v, 0); }

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

// What the warps that add take over: the TMEM address of the thread's first
// column, the distance of the halves, the tokens' scales of block of k `it` (a
// ring of `kept`), the barrier that gives the accumulator back.
struct Handover {
  uint32_t from, widest;
  const float* scales;
  uint32_t it, kept;
  uint64_t *empty, *next;  // ... and the one that hands over the next
  uint32_t next_parity;
};

// How a warp reads a block of k of up to kOf chunks of 16 tokens.  Its columns are
// octets of 8 tokens in planes of 16 weight rows: in the plain product two planes
// (the warp's 32 rows) of 2 kOf octets, in SwiGLU four (the gate's, then the up
// projection's) of kOf, as a warp takes half of the tokens there.  Of an octet and
// a plane a thread has four numbers: two weight rows by two tokens, the same two of
// eight at every octet, so that all its rows share a pair of scales an octet.
// (With a weight row a thread, every thread took every scale from shared memory:
// swiglu decode 103 us instead of 96, prefill 949 instead of 834.)
// An item is 16 registers: as many octets of a plane as one load brings, since
// each load takes some 18 cycles to issue whatever it brings.
template <bool kSwiglu, int kOf>
struct Plan {
  static constexpr int kPlanes = kSwiglu ? 4 : 2, kOctets = kSwiglu ? kOf : 2 * kOf;
  static constexpr int kItems = kOf == kChunks ? 8 : kOf;  // of a block of k
  static constexpr int kBlocks = kOf == 1 ? 4 : kOf == kChunks ? 1 : 2;  // blocks of k in a hand-over, at most
  static constexpr int kMost = kItems * kBlocks;
  // octets that one load of item i brings, and the plane and octet of its g-th four registers
  __host__ __device__ static constexpr int load(int i) {
    return kOf == kChunks ? 4 : kOf == 3 ? (i < 2 ? kPlanes == 2 ? 4 : 2 : kPlanes == 2 ? 2 : 1) : kOctets;
  }
  __host__ __device__ static constexpr int plane(int i, int g) {
    return kOf == kChunks ? i % kPlanes : (kOf == 3 && i == 2 ? 0 : i * (4 / load(i))) + g / load(i);
  }
  __host__ __device__ static constexpr int octet(int i, int g) {
    return kOf == kChunks ? i / kPlanes * 4 + g : (kOf == 3 && i == 2 ? load(0) : 0) + g % load(i);
  }
};

template <bool kSwiglu, int kOf, int kItem, int kLoad = 0>
__device__ __forceinline__ void load_planes(uint32_t (&v)[16], uint32_t from, uint32_t widest) {
  using P = Plan<kSwiglu, kOf>;
  constexpr int kOctets = P::load(kItem), g = kLoad * kOctets;
  if constexpr (g < 4) {
    constexpr int plane = P::plane(kItem, g);
    constexpr uint32_t at = 8 * P::octet(kItem, g) + ((plane & 1) << 20);  // sixteen lanes on: 16 << 16
    tmem_load_octets<kOctets>(from + at + (plane >> 1) * widest, v + 4 * g);
    load_planes<kSwiglu, kOf, kItem, kLoad + 1>(v, from, widest);
  }
}

// Item m of a hand-over: item m % kItems of its (m / kItems)th block of k.
template <bool kSwiglu, int kOf, int m>
__device__ __forceinline__ void load_item(uint32_t (&v)[4][16], const Handover& h, int items) {
  constexpr int kItems = Plan<kSwiglu, kOf>::kItems;
  if (m < items) load_planes<kSwiglu, kOf, m % kItems>(v[m & 3], h.from + (m / kItems) * 2 * h.widest, h.widest);
}

template <bool kSwiglu, int kOf, int m>
__device__ __forceinline__ void add_item(float (&acc)[16 * kOf], const uint32_t (&v)[4][16],
                                         const float2 (&scales)[Plan<kSwiglu, kOf>::kBlocks][Plan<kSwiglu, kOf>::kOctets],
                                         int items) {
  using P = Plan<kSwiglu, kOf>;
  if (m >= items) return;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int plane = P::plane(m % P::kItems, g), octet = P::octet(m % P::kItems, g);
    if (octet >= P::kOctets) continue;
    const float2 s = scales[m / P::kItems][octet];
#pragma unroll
    for (int r = 0; r < 4; r += 2) {
      float* a = acc + (octet * P::kPlanes + plane) * 4 + r;
      const uint32_t* f = v[m & 3] + 4 * g + r;
      const float2 sum = fma2(make_float2(__uint_as_float(f[0]), __uint_as_float(f[1])), s, make_float2(a[0], a[1]));
      a[0] = sum.x, a[1] = sum.y;
    }
  }
}

__device__ __forceinline__ void release(const Handover& h) {
  tmem_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(h.empty);
}

// Registers of loads that the wait for others has settled.
__device__ __forceinline__ void settled(uint32_t* v) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// Whether a barrier's phase is complete, without waiting.
__device__ __forceinline__ bool phase_over(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done)
               : "r"(bar), "r"(parity)
               : "memory");
  return done != 0;
}

// Adds a hand-over's `blocks` blocks of k, `items` items: 64 registers' loads are on
// their way at a time, and the accumulator goes back as soon as the last are here.
// Returns whether the next hand-over is there already, asked for before the last
// sums, since the answer takes as long as they do (decode 51.0 -> 49.9 us; where a
// hand-over fills the registers, one more costs spills: prefill 596 -> 748 us).
template <bool kSwiglu, int kOf>
__device__ __forceinline__ bool take(float (&acc)[16 * kOf], const Handover& h, int blocks, int items) {
  using P = Plan<kSwiglu, kOf>;
  uint32_t v[4][16];
  load_item<kSwiglu, kOf, 0>(v, h, items), load_item<kSwiglu, kOf, 1>(v, h, items);
  load_item<kSwiglu, kOf, 2>(v, h, items), load_item<kSwiglu, kOf, 3>(v, h, items);
  // scales of rows past the group's end are anything
  float2 scales[P::kBlocks][P::kOctets];
#pragma unroll
  for (int k = 0; k < P::kBlocks; ++k) {
    if (k && k >= blocks) continue;
    const float2* f = reinterpret_cast<const float2*>(h.scales + ((h.it + k) & (h.kept - 1)) * h.widest);
#pragma unroll
    for (int o = 0; o < P::kOctets; ++o) scales[k][o] = f[4 * o];
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) m ? settled(v[m]) : tmem_load_wait16(v[m]);
  bool next = false;
  if (P::kMost <= 4 || items <= 4) {
    release(h);
    if constexpr (kOf != kChunks) next = phase_over(smem_u32(h.next), h.next_parity);
    add_item<kSwiglu, kOf, 0>(acc, v, scales, items), add_item<kSwiglu, kOf, 1>(acc, v, scales, items);
    add_item<kSwiglu, kOf, 2>(acc, v, scales, items), add_item<kSwiglu, kOf, 3>(acc, v, scales, items);
  } else if constexpr (P::kMost > 4) {
    add_item<kSwiglu, kOf, 0>(acc, v, scales, items), load_item<kSwiglu, kOf, 4>(v, h, items);
    add_item<kSwiglu, kOf, 1>(acc, v, scales, items), load_item<kSwiglu, kOf, 5>(v, h, items);
    add_item<kSwiglu, kOf, 2>(acc, v, scales, items);
    if constexpr (P::kMost > 6) load_item<kSwiglu, kOf, 6>(v, h, items);
    add_item<kSwiglu, kOf, 3>(acc, v, scales, items);
    if constexpr (P::kMost > 6) load_item<kSwiglu, kOf, 7>(v, h, items);
#pragma unroll
    for (int m = 4; m < P::kMost; ++m) m > 4 ? settled(v[m & 3]) : tmem_load_wait16(v[m & 3]);
    release(h);
    if constexpr (kOf != kChunks) next = phase_over(smem_u32(h.next), h.next_parity);
    add_item<kSwiglu, kOf, 4>(acc, v, scales, items), add_item<kSwiglu, kOf, 5>(acc, v, scales, items);
    if constexpr (P::kMost > 6)
      add_item<kSwiglu, kOf, 6>(acc, v, scales, items), add_item<kSwiglu, kOf, 7>(acc, v, scales, items);
  }
  return next;
}

// What all warps know of the launch.
struct Launch {
  uint32_t tmem, widest, acc_columns, kept;
  int per, tiles_n, blocks_k;
  unsigned tiles;
};

// The warps that add, in a launch whose tiles have up to kOf chunks of 16 tokens.
template <bool kSwiglu, int kOf>
__device__ __forceinline__ void add_tiles(const Matmul4Args& p, Shared& s, const unsigned* prefix, const Launch& l) {
  constexpr int kColumns = 16 * kOf;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = warp >> 2, quarter = warp & 3;
  const int pair = 2 * (lane & 3);                        // the thread's columns of eight
  volatile int* quit = &s.quit;
  int* err = p.groups.err;
  const int F = p.N >> 1;
  uint32_t it = 0, group = 0;  // blocks of k and hand-overs of all tiles
  int turn = 0;
  bool ok = true, ready = false;  // whether the next hand-over is there
  for (unsigned t = blockIdx.x; t < l.tiles; t += gridDim.x, turn ^= 1) {
    const Tile c = tile_at(p.groups, prefix, l.tiles_n, t);
    // a warp's columns: all of its half's, or half of both halves' (SwiGLU: 8
    // tokens' gates, then their up projections)
    const int first = kSwiglu ? half * (c.columns >> 1) : 0;
    const uint32_t from = l.tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (kSwiglu ? first : half * l.widest);
    float acc[kColumns];
#pragma unroll
    for (int j = 0; j < kColumns; ++j) acc[j] = 0.0f;
    for (int kb = 0; kb < l.blocks_k; ++group) {
      const uint32_t ac = group & 1;
      const int n = min(l.per, l.blocks_k - kb);
      // no vote a hand-over (prefill 579 -> 560 us): the tile's end has one
      ok = ok && (ready || wait_or_quit(&s.acc_full[ac], (group >> 1) & 1, quit, err));
      __syncwarp();
      tmem_fence_after();
      const Handover h{from + ac * l.acc_columns, l.widest, s.x_scale + first + pair, it, l.kept, &s.acc_empty[ac],
                       &s.acc_full[ac ^ 1], ((group + 1) >> 1) & 1};
      using P = Plan<kSwiglu, kOf>;
      ready = take<kSwiglu, kOf>(acc, h, n, kOf == kChunks ? (c.columns + 16 * P::kPlanes - 1) / (16 * P::kPlanes) * P::kPlanes : n * kOf);
      kb += n;
      it += n;
    }
    if (!__all_sync(kFullMask, ok)) return;
    if constexpr (!kSwiglu) {
      // Lanes 4 a + t hold weight rows a, a + 8, a + 16 and a + 24 of the same tokens.
      // Four of them swap theirs, so that each has four rows in a row, 8 bytes.
      const int a = lane >> 2;
      const int n = c.n * 256 + half * 128 + quarter * 32 + 8 * (a & 3) + (a & 4);
      uint16_t* o = p.out + (c.row + pair) * p.N + n;
      const int rows = n < p.N ? c.rows - pair : 0;
#pragma unroll
      for (int i = 0; i < kColumns / 4; ++i) {
        const float* v = acc + 8 * (i >> 1) + (i & 1);  // token 8 (i / 2) + pair + i % 2
        const uint32_t w0 = pack_bf16x2(v[0], v[2]), w1 = pack_bf16x2(v[4], v[6]);
        const uint32_t x = __shfl_xor_sync(kFullMask, __byte_perm(w0, w1, a & 1 ? 0x5410 : 0x7632), 4);
        const uint32_t u0 = a & 1 ? __byte_perm(w0, x, 0x3254) : __byte_perm(w0, x, 0x5410);
        const uint32_t u1 = a & 1 ? __byte_perm(w1, x, 0x3276) : __byte_perm(w1, x, 0x7610);
        const uint32_t y = __shfl_xor_sync(kFullMask, a & 2 ? u0 : u1, 8);
        const int token = 8 * (i >> 1) + (i & 1);
        if (token < rows)
          *reinterpret_cast<uint2*>(o + static_cast<long long>(token) * p.N) = a & 2 ? make_uint2(y, u1) : make_uint2(u0, y);
      }
    } else {
      const int live = c.rows - first;  // of this warp's tokens (and more, where the other half has some)
      const long long row = c.row + first;
      float (*amax)[4] = s.amax[turn][half];
      // the weights of all its tokens are on their way together
      float w[2 * kOf];
#pragma unroll
      for (int i = 0; i < 2 * kOf; ++i) {
        const int token = 8 * (i >> 1) + pair + (i & 1);
        w[i] = p.row_weights && token < min(live, c.columns >> 1) ? p.row_weights[row + token] : 1.0f;
      }
#pragma unroll
      for (int i = 0; i < 2 * kOf; ++i) {
        // token 8 (i / 2) + pair + i % 2: its four weight rows of this thread
        const int token = 8 * (i >> 1) + pair + (i & 1);
        float most = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float& g = acc[16 * (i >> 1) + 2 * r + (i & 1)];
          const float u = acc[16 * (i >> 1) + 8 + 2 * r + (i & 1)];
          g = __fdividef(g, 1.0f + __expf(-g)) * u * w[i];
          most = fmaxf(most, fabsf(g));  // a NaN does not enter the maximum
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) most = fmaxf(most, __shfl_xor_sync(kFullMask, most, d));
        if (lane < 4) amax[token][quarter] = most;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.amax_full[half]);
      ok = __all_sync(kFullMask, wait_or_quit(&s.amax_full[half], turn, quit, err));
      if (!ok) return;
      // Lanes 4 a + t: a byte of weight rows a, a + 8, a + 16 and a + 24 each.  Four
      // lanes swap theirs, so that each has four rows in a row.
      const int a = lane >> 2;
      unsigned char* o = p.act.data + row * F + c.n * 128 + quarter * 32 + 8 * (a & 3) + (a & 4);
      const int mine = min(live, c.columns >> 1);
      // a lane's tokens' scales and their inverses: two divisions for each, not in every lane
      float* inv = s.inv[half][quarter];
#pragma unroll 1
      for (int token = lane; token < 8 * kOf; token += 32) {
        const float4 m = *reinterpret_cast<const float4*>(amax[token]);
        const float sc = group_scale(fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w)), &inv[token]);
        if (quarter == 0 && token < mine) *p.act.scale(row + token, c.n) = sc;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2 * kOf; ++i) {
        const int token = 8 * (i >> 1) + pair + (i & 1);
        float q[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) q[r] = acc[16 * (i >> 1) + 2 * r + (i & 1)];
        uint32_t v = quant4(q, inv[token]);
        uint32_t x = __shfl_xor_sync(kFullMask, v, 4);
        v = a & 1 ? __byte_perm(v, x, 0x3715) : __byte_perm(v, x, 0x6240);
        x = __shfl_xor_sync(kFullMask, v, 8);
        v = a & 2 ? __byte_perm(v, x, 0x3276) : __byte_perm(v, x, 0x5410);
        if (token < mine) *reinterpret_cast<uint32_t*>(o + static_cast<long long>(token) * F) = v;
      }
    }
  }
}

}  // namespace

template <bool kSwiglu>
__global__ void __launch_bounds__(kThreads, 1)
    k_grouped_matmul_w4(const __grid_constant__ Matmul4Maps maps, const Matmul4Args p, uint32_t smem_bytes) {
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
    for (int i = 0; i < 2; ++i) mbar_init(&s.acc_empty[i], kEpilogueWarps), mbar_init(&s.amax_full[i], 4), mbar_init(&s.drained[i], 1);
    s.quit = 0;
    s.columns = 16;
    mbar_init_fence();
    prefetch_map(&maps.x[0]);
    prefetch_map(&maps.scales);
    prefetch_map(&maps.w);
  }
  if (warp == kEpilogueWarps + 1) tmem_alloc(&s.tmem, kTmemColumns);
  __syncthreads();
  after_previous();
  groups_prefix(p.groups, kTileT, prefix, s.sums,
                [&](int n) { if (n) atomicMax(&s.columns, rows_per_tile(n, (n + kTileT - 1) / kTileT)); });
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = uniform(s.tmem);
  // As many stages as fit beside the largest tile's tokens; an accumulator holds
  // several blocks of k where the tiles have few.
  const uint32_t widest = uniform(s.columns);
  const uint32_t stage_bytes = kTokens + widest * kBlockK;
  const int per = widest <= 16 ? 4 : widest <= 48 ? 2 : 1;
  // A wait for a stage tells its rounds apart by parity, so the round before has to be
  // over by then.  With an even number of stages the same issuing warp has waited for
  // it.  With an odd one the other has, and the accumulators' waits have to say it: that all
  // before the last hand-over is done (or, per == 1, where the stage is waited for
  // first, before the last three).
  const uint32_t fit = min(static_cast<uint32_t>(kMaxStages), (smem_bytes - static_cast<uint32_t>(stages - raw)) / stage_bytes);
  const uint32_t num_stages = (fit & 1) && (per == 4 || fit < 5) ? fit - 1 : fit;
  const uint32_t acc_columns = per * 2 * widest;
  const uint32_t kept = per == 1 ? 16 : 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&s.acc_full[i], per);
    mbar_init_fence();
  }
  // the tokens' scales inside the MMA are 2^0: theirs are applied behind it
  if (warp < 4) tmem_fill4(tmem + (static_cast<uint32_t>(warp * 32) << 16) + kTokenScales, 0x7f7f7f7fu);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();

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
        const int row = uniform(static_cast<uint32_t>(c.row)), columns = uniform(c.columns), n = uniform(c.n), g = uniform(c.group);
        for (int kb = 0; kb < blocks_k; ++kb, ++it) {
          if (it >= num_stages) {
            ok = __all_sync(kFullMask, wait_or_quit(&s.empty[st], phase ^ 1, quit, err));
            if (!ok) break;
          }
          if (elect_one()) {
            unsigned char* a = stages + st * stage_bytes;
            unsigned char* f = a + 2 * kHalfBytes;
            unsigned char* b = a + kTokens;
            uint64_t* bar = &s.full[st];
            mbar_arrive_expect_tx(bar, 2 * (kHalfLoad + kScaleBytes) + columns * kBlockK);
            if constexpr (kSwiglu) {
              tma_load_4d(a, &maps.w, kb * kBlockK, n * 128, 0, g, bar);
              tma_load_3d(f, &maps.scales, kb * (kScaleBytes / 4), n, g * 2, bar);
            } else {
              tma_load_3d(a, &maps.w, kb * kBlockK, n * 256, g, bar);
              tma_load_2d(f, &maps.scales, kb * (kScaleBytes / 4), g * blocks_n + 2 * n, bar);
            }
            int y = row;
#pragma unroll
            for (int i = 2; i >= 0; --i) {
              if (columns & (16 << i)) {
                tma_load_2d(b, &maps.x[i], kb * kBlockK, y, bar);
                b += (16 << i) * kBlockK;
                y += 16 << i;
              }
            }
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
      const uint32_t b_scales = tmem + kTokenScales;
      uint32_t it = 0, st = 0, phase = 0, group = 0;  // of all tiles: blocks of k, their stage, hand-overs
      bool ok = true;
      for (unsigned t = blockIdx.x; __all_sync(kFullMask, ok) && t < tiles; t += gridDim.x) {
        const Tile c = tile_at(p.groups, prefix, tiles_n, t);
        const uint32_t desc = mma_mx_desc(128, uniform(c.columns), 0);
        for (int kb = 0, in = 0; kb < blocks_k; ++kb, ++it) {
          const uint32_t at = st, round = phase, ac = group & 1, turn = (group >> 1) & 1, slot = in;
          const bool last = kb + 1 == blocks_k;
          if (++st == num_stages) st = 0, phase ^= 1;
          if (++in == per || last) in = 0, ++group;
          if ((it & 1) != odd) continue;
          // With many tokens the operands first, which are here long before the accumulator
          // is back, and no vote: all of it is on the accumulators' round (prefill 605 ->
          // 575 us).  (A fresh barrier counts as having ended the round before its first.)
          uint64_t *wait1 = &s.acc_empty[ac], *wait2 = &s.full[at];
          uint32_t parity1 = turn ^ 1, parity2 = round;
          if (per == 1) {
            wait1 = &s.full[at], wait2 = &s.acc_empty[ac];
            parity1 = round, parity2 = turn ^ 1;
          }
          ok = ok && wait_or_quit(wait1, parity1, quit, err) && wait_or_quit(wait2, parity2, quit, err);
          __syncwarp();
          tmem_fence_after();
          if (elect_one() && ok) {
            // descriptors count 16-byte units; 32 channels are two
            const uint64_t a = first + at * (stage_bytes >> 4), b = a + (kTokens >> 4);
            const uint64_t f = first_scales + at * (stage_bytes >> 4);
            const uint32_t d = tmem + ac * acc_columns + slot * 2 * widest;
            const uint32_t a_scales = tmem + 2 * acc_columns + (ac * per + slot) * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) tmem_copy_scales(a_scales + 4 * h, f + h * (kScaleBytes >> 4));
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_mx(d + h * widest, a + h * (kHalfBytes >> 4) + 2 * j, b + 2 * j,
                       desc | (static_cast<uint32_t>(j) << 4) | (static_cast<uint32_t>(j) << 29), a_scales + 4 * h,
                       b_scales, j > 0);
            // the last hand-over of a tile may hold fewer blocks than the barrier counts
            if (last)
              for (int i = slot + 1; i < per; ++i) mbar_arrive(&s.acc_full[ac]);
            mma_commit(&s.acc_full[ac]);
            mma_commit(&s.empty[at]);
          }
          __syncwarp();
        }
      }
      // nor may an MMA: all are done before TMEM goes back
      int none = 0;
      if (elect_one()) mma_commit(&s.drained[odd]);
      __syncwarp();
      wait_or_quit(&s.drained[odd], 0, &none, err);
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
          const uint32_t dst = smem_u32(&s.x_scale[(it % kept) * widest + lane]);
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
    const Launch l{tmem, widest, acc_columns, kept, per, tiles_n, blocks_k, tiles};
    if (widest <= 16)
      add_tiles<kSwiglu, 1>(p, s, prefix, l);
    else if (widest <= 32)
      add_tiles<kSwiglu, 2>(p, s, prefix, l);
    else if (widest <= 48)
      add_tiles<kSwiglu, 3>(p, s, prefix, l);
    else
      add_tiles<kSwiglu, kChunks>(p, s, prefix, l);
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
  const bool swiglu = p.act.data != nullptr;
  Matmul4Maps maps;
  cudaError_t e = cudaSuccess;
  for (int i = 0; e == cudaSuccess && i < 3; ++i) e = make_byte_map(&maps.x[i], p.x.data, p.K, p.groups.rows, 0, 16 << i);
  if (e != cudaSuccess) return e;
  const cuuint64_t K = p.K, N = p.N, G = p.groups.G, blocks_n = (N + 127) / 128, row = K / 128 * kScaleBytes;
  if (swiglu) {
    // both halves at once: the gate's rows, then the up projection's
    const cuuint64_t dims[4] = {K, N / 2, 2, G}, strides[3] = {K / 2, N / 2 * (K / 2), N * (K / 2)};
    const cuuint32_t box[4] = {kBlockK, 128, 2, 1};
    e = make_tensor_map(&maps.w, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, p.w, 4, dims, strides, box, true);
    const cuuint64_t sdims[3] = {row / 4, blocks_n / 2, 2 * G}, sstrides[2] = {row, row * (blocks_n / 2)};
    const cuuint32_t sbox[3] = {kScaleBytes / 4, 1, 2};
    if (e == cudaSuccess)
      e = make_tensor_map(&maps.scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, p.w_scales, 3, sdims, sstrides, sbox, false);
  } else {
    const cuuint64_t dims[3] = {K, N, G}, strides[2] = {K / 2, N * (K / 2)};
    const cuuint32_t box[3] = {kBlockK, 256, 1};
    e = make_tensor_map(&maps.w, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, p.w, 3, dims, strides, box, true);
    const cuuint64_t sdims[2] = {row / 4, blocks_n * G}, sstrides[1] = {row};
    const cuuint32_t sbox[2] = {kScaleBytes / 4, 2};
    if (e == cudaSuccess)
      e = make_tensor_map(&maps.scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, p.w_scales, 2, sdims, sstrides, sbox, false);
  }
  if (e != cudaSuccess) return e;
  int device = 0, smem = 0;  // all of it: the kernel decides on the stages
  if ((e = cudaGetDevice(&device)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, device)) != cudaSuccess)
    return e;
  const size_t least = sizeof(Shared) + sizeof(unsigned) * (p.groups.G + 1) + 1023 + 2 * (kTokens + kTileT * kBlockK);
  if (least > static_cast<size_t>(smem)) return cudaErrorInvalidValue;
  auto kernel = swiglu ? k_grouped_matmul_w4<true> : k_grouped_matmul_w4<false>;
  static std::atomic<unsigned long long> ready[2];  // devices set up, a bit each
  if ((e = set_up_kernel(reinterpret_cast<const void*>(kernel), ready[swiglu], kLaunchRegisters)) != cudaSuccess) return e;
  return launch_early(kernel, 1, dim3(sms), dim3(kThreads), smem, stream, maps, p,
                      static_cast<uint32_t>(smem));
}

}  // namespace ep
