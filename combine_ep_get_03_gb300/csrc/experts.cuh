// What the experts' kernels share: groups of rows as dispatch leaves them,
// e4m3 rows with a scale for every 128 channels, and waits that end.
#pragma once

#include <atomic>

#include "device_common.cuh"
#include "ep_internal.h"

namespace ep {

constexpr int kMaxGroups = 4096;
constexpr int kTile4Rows = 112;  // rows of a tile of the products on 4-bit weights

// Groups of rows: group g holds count[g] rows from offset[g], or from
// g * rows_per_group where offset is null.
struct GroupArgs {
  const int* count;
  const int* offset;
  int G;
  long long rows;            // rows of every row buffer
  long long rows_per_group;  // with offset null
  int* err;                  // status word or null
};

// e4m3 rows: the scale of row r, channels [128 g, 128 g + 128) is
// scales[r * row_stride + g * group_stride].
struct Fp8Rows {
  unsigned char* data;
  float* scales;
  long long row_stride, group_stride;
  __device__ __forceinline__ float* scale(long long r, int g) const {
    return scales + r * row_stride + g * group_stride;
  }
};

__device__ __forceinline__ void latch_status(int* err, int code) {
  if (err) latch_error(err, code);
}

// Waits until the stream's earlier kernels have ended and their results are
// visible, then lets a kernel launched the same way start its own preparations
// (barriers, TMEM) on SMs that become free.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" : : : "memory");
  asm volatile("griddepcontrol.launch_dependents;" : : : "memory");
}

// First row and row count of group g.  A group that does not fit its slots or
// the row buffer is cut to what does (EP_ERR_CAPACITY, latched by `report`).
__device__ __forceinline__ int group_span(const GroupArgs& a, int g, long long* start, bool report) {
  const long long first = a.offset ? static_cast<long long>(a.offset[g]) : g * a.rows_per_group;
  long long n = a.count[g];
  long long most = a.offset ? a.rows - first : a.rows_per_group;
  if (first < 0 || most < 0) most = 0;
  if (n < 0) n = 0;
  if (n > most) {
    n = most;
    if (report) latch_status(a.err, kErrCapacity);
  }
  *start = first;
  return static_cast<int>(n);
}

// prefix[g] = tiles of `tile_rows` rows in the groups before g, prefix[G] =
// all of them, for the whole block; `sums` holds 32 words.  Groups that do not
// overlap have rows / tile_rows + G tiles at most; counts that say more are cut
// there (EP_ERR_CAPACITY), which also keeps prefix[G] times the column tiles,
// bounded by the host for that many, within 32 bits.  `each` sees every group's
// row count, in some thread.
template <typename Each>
__device__ __forceinline__ void groups_prefix(const GroupArgs& a, int tile_rows, unsigned* prefix, unsigned* sums,
                                              Each each) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int per = (a.G + blockDim.x - 1) / blockDim.x;
  const int g0 = tid * per;
  const unsigned most = static_cast<unsigned>(a.rows / tile_rows) + a.G;
  auto add = [most](unsigned x, unsigned y) {
    const unsigned s = x + y;
    return s < x || s > most ? most + 1 : s;
  };
  unsigned mine = 0;
  for (int g = g0; g < g0 + per && g < a.G; ++g) {
    long long first;
    const int n = group_span(a, g, &first, blockIdx.x == 0);
    each(n);
    const unsigned t = static_cast<unsigned>((static_cast<long long>(n) + tile_rows - 1) / tile_rows);
    prefix[g] = t;
    mine = add(mine, t);
  }
  unsigned incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned v = __shfl_up_sync(kFullMask, incl, d);
    if (lane >= d) incl = add(incl, v);
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  unsigned base = 0, all = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) base = add(base, sums[w]);
    all = add(all, sums[w]);
  }
  unsigned before = __shfl_up_sync(kFullMask, incl, 1);
  before = add(base, lane ? before : 0u);
  for (int g = g0; g < g0 + per && g < a.G; ++g) {
    const unsigned t = prefix[g];
    prefix[g] = before;
    before = add(before, t);
  }
  if (tid == 0) {
    prefix[a.G] = all;
    if (all > most && blockIdx.x == 0) latch_status(a.err, kErrCapacity);
  }
  __syncthreads();
}

__device__ __forceinline__ void groups_prefix(const GroupArgs& a, int tile_rows, unsigned* prefix, unsigned* sums) {
  groups_prefix(a, tile_rows, prefix, sums, [](int) {});
}

// The group that item i (< prefix[G]) belongs to.
__device__ __forceinline__ int find_group(const unsigned* prefix, int G, unsigned i) {
  int lo = 0, hi = G;  // prefix[lo] <= i < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// Bounded wait on an mbarrier phase for kernels whose warps wait on one
// another: one that gives up latches EP_ERR_TIMEOUT and raises `quit`, which
// ends every other warp's wait too.
// `kCluster`: the barrier's arrivals may come from the cluster's other block.
template <bool kCluster>
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  uint32_t done;
  if (kCluster)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
  return done != 0;
}
template <bool kCluster = false>
__device__ __forceinline__ bool wait_or_quit(uint64_t* bar, uint32_t parity, volatile int* quit, int* err) {
  const uint32_t addr = smem_u32(bar);
  if (phase_done<kCluster>(addr, parity)) return true;
  for (int it = 0; it < kSpinLimit; ++it) {
    if (phase_done<kCluster>(addr, parity)) return true;
    if (it >= 64) {
      if (*quit) return false;
      __nanosleep(32);
    }
  }
  *quit = 1;
  latch_status(err, kErrTimeout);
  return false;
}

// 32 bytes from registers, as one store where the address allows it.
__device__ __forceinline__ void store32(void* p, const uint32_t* v, bool aligned32) {
  if (aligned32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :
                 : "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Four e4m3 codes of one word as fp32 (exact).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* f) {
  uint32_t lo, hi;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n" : "=f"(f[0]), "=f"(f[1]) : "r"(lo));
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n" : "=f"(f[2]), "=f"(f[3]) : "r"(hi));
}

// Four fp32 -> four e4m3 codes, each the saturating nearest-even image of x * inv.
__device__ __forceinline__ uint32_t quant4(const float* x, float inv) {
  return pack_e4m3x2(x[0] * inv, x[1] * inv) | (pack_e4m3x2(x[2] * inv, x[3] * inv) << 16);
}

// A 128-channel group's scale and inverse from its largest magnitude, as
// dispatch quantises: a = max(amax, 1e-4), scale = a / 448, inv = 448 / a.
__device__ __forceinline__ float group_scale(float amax, float* inv) {
  const float a = fmaxf(amax, 1e-4f);
  *inv = __fdiv_rn(448.0f, a);
  return __fdiv_rn(a, 448.0f);
}

// ------------------------------------------------------------------ launches

// Launch that may begin while the stream's previous kernel ends: the kernel
// calls after_previous() before it touches any memory but its own.  `cluster`
// blocks form a cluster.  Back to back this saves about 2 us a call (one
// token's product 45.2 -> 43.3 us, a small weight gradient 15.7 -> 14.2 us).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_early(void (*kernel)(KArgs...), int cluster, dim3 grid, dim3 block, size_t smem,
                                cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Once per kernel and device: the whole shared memory for dynamic use, and the
// register count that a kernel moving registers between warps relies on.
inline cudaError_t set_up_kernel(const void* kernel, std::atomic<unsigned long long>& ready, int registers) {
  int device = 0, optin = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (device & 63);
  if (device < 64 && (ready.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  if (registers) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
    if (fa.numRegs < registers) return cudaErrorInvalidValue;
  }
  if ((e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device)) != cudaSuccess) return e;
  if ((e = set_dynamic_smem_limit(kernel, 0, optin)) != cudaSuccess) return e;
  if (device < 64) ready.fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

struct GateArgs {
  const void* logits;  // [T][ld] fp32 or bf16
  long long ld;
  const uint8_t* mask;  // [T] or null: 0 = padding token
  int T, E, k, groups, keep, sigmoid, ids32;
  int vec;  // rows readable as 16-byte words (grad_vec: writable)
  float coef;
  float fixed;     // 1 / step of the blocks' probability sums
  void* idx;       // [T][k]
  float* weights;  // [T][k]
  int* count;      // [E + 1]
  float* prob;     // [E]
  float* loss;     // [1]
  unsigned* work;  // zeroed; left zeroed
  // backward
  const float* grad_weights;  // [T][k] or null
  const float* grad_loss;     // [1] or null
  void* grad_logits;          // [T][grad_ld], the logits' type
  long long grad_ld;
  int grad_vec;
};

struct SwigluBackwardArgs {
  GroupArgs groups;
  const uint16_t* grad_act;  // bf16 [rows][F]
  Fp8Rows pre;               // [rows][2F]
  const float* row_weights;  // [rows] or null
  Fp8Rows grad_pre;          // [rows][2F]
  float* grad_row_weights;   // [rows] or null
  int F;
};

// One grouped product; act.data selects the SwiGLU epilogue (N = 2F then).
struct MatmulArgs {
  GroupArgs groups;
  Fp8Rows x;             // [rows][K]
  const void* w;         // e4m3 [G][N][K]
  const float* w_scales; // [G][ceil(N/128)][K/128]
  int N, K;
  uint16_t* out;            // bf16 [rows][N], or null
  Fp8Rows act;              // [rows][F]
  Fp8Rows pre;              // [rows][2F], data null if not kept
  const float* row_weights; // [rows] or null
};

// The same products on 4-bit weights; act.data selects the SwiGLU epilogue.
struct Matmul4Args {
  GroupArgs groups;
  Fp8Rows x;                      // [rows][K]
  const void* w;                  // e2m1 [G][N][K/2], two codes a byte
  const unsigned char* w_scales;  // [G][ceil(N/128)][K/128][512]
  int N, K;
  uint16_t* out;            // bf16 [rows][N], or null
  Fp8Rows act;              // [rows][F]
  const float* row_weights; // [rows] or null
};

// dw[g] = sum over the group's rows of dy^T x.
struct WeightGradArgs {
  GroupArgs groups;
  Fp8Rows dy;  // [rows][N]
  Fp8Rows x;   // [rows][K]
  int N, K;
  uint16_t* dw;  // bf16 [G][N][K]
};

cudaError_t launch_gate(const GateArgs& p, bool bf16, bool backward, int sms, cudaStream_t stream);
cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& p, int sms, cudaStream_t stream);
cudaError_t launch_grouped_matmul(const MatmulArgs& p, int sms, cudaStream_t stream);
cudaError_t launch_grouped_matmul_w4(const Matmul4Args& p, int sms, cudaStream_t stream);
cudaError_t launch_weight_grad(const WeightGradArgs& p, int sms, cudaStream_t stream);
size_t gate_work_bytes(int E);
// out[i] = row_weights[the expert-major row of entry i], 0 where masked.
cudaError_t launch_em_combine_weights(const int* idx, const int* slot, const int* offset, const float* row_weights,
                                      long long rows, long long entries, float* out, int* err, cudaStream_t stream);

}  // namespace ep
