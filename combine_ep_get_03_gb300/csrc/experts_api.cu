// C ABI of the experts' side (include/ep.h): argument checks and launch
// configuration of the gate, the grouped products, the SwiGLU backward and the
// weight gradient.  None needs a handle; every result goes to caller buffers.
#include <climits>
#include <cstdio>
#include <cstdlib>

#include "block_norm.cuh"
#include "ep.h"
#include "ep_internal.h"
#include "experts.cuh"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

ep_status_t status_of(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return EP_OK;
  if (std::getenv("EP_DEBUG")) std::fprintf(stderr, "[ep] %s: %s\n", what, cudaGetErrorString(e));
  return EP_ERR_CUDA;
}

// SMs to occupy on the current device.
ep_status_t sm_count(int num_sms, int* out) {
  int device = 0, n = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return status_of(e, "device");
  *out = num_sms <= 0 || num_sms > n ? n : num_sms;
  return EP_OK;
}

bool groups_ok(const ep_groups_t* g) {
  if (!g || g->num_groups < 1 || g->num_groups > ep::kMaxGroups || !g->count || !aligned(g->count, 4) ||
      (g->offset && !aligned(g->offset, 4)) || (g->status && !aligned(g->status, 4)) || g->rows < 0 || g->rows > INT_MAX)
    return false;
  return g->offset || (g->rows_per_group >= 0 && g->rows_per_group <= INT_MAX &&
                       g->rows_per_group * g->num_groups <= g->rows);
}

// Tiles of a product over `rows` rows are counted in 32 bits (one more than
// the groups can have where counts overlap).
bool tiles_ok(const ep_groups_t* g, int N) {
  return (g->rows / 128 + g->num_groups + 1) * ((N + 127) / 128) < INT_MAX / 2;
}

ep::GroupArgs groups_of(const ep_groups_t* g) {
  return ep::GroupArgs{g->count, g->offset, g->num_groups, g->rows, g->offset ? 0 : g->rows_per_group, g->status};
}

bool rows_ok(const ep_fp8_rows_t* r) {
  return r && r->data && r->scales && aligned(r->data, 16) && aligned(r->scales, 4) && r->row_stride >= 0 &&
         r->group_stride >= 0;
}

ep::Fp8Rows rows_of(const ep_fp8_rows_t* r) {
  return ep::Fp8Rows{static_cast<unsigned char*>(r->data), r->scales, r->row_stride, r->group_stride};
}

bool gate_ok(const void* logits, ep_logits_t type, int64_t ld, int T, int E, int k, ep_gate_score_t score) {
  if ((type != EP_LOGITS_FP32 && type != EP_LOGITS_BF16) || (score != EP_GATE_SOFTMAX && score != EP_GATE_SIGMOID))
    return false;
  if (T < 0 || T > (1 << 26) || E < 1 || E > 4096 || k < 1 || k > 32 || k > E || ld < E) return false;
  return T == 0 || (logits && aligned(logits, type == EP_LOGITS_FP32 ? 4 : 2));
}

// Whether rows of logits split into 16-byte words.
bool words16(const void* p, ep_logits_t type, int64_t ld, int E) {
  const int per = type == EP_LOGITS_FP32 ? 4 : 8;
  return E % per == 0 && ld % per == 0 && aligned(p, 16);
}

bool norm_ok(const ep_block_norm_t* n) {
  return n && n->num_tokens >= 0 && n->hidden >= 8 && n->hidden % 8 == 0 && n->hidden <= ep::kBlockNormMaxHidden &&
         (n->residual_type == EP_REAL_FP32 || n->residual_type == EP_REAL_BF16) &&
         (n->weight_type == EP_REAL_FP32 || n->weight_type == EP_REAL_BF16) && aligned(n->post_weight, 16) &&
         aligned(n->pre_weight, 16) && aligned(n->gate, 16);
}

ep::BlockNormArgs norm_args(const ep_block_norm_t* n) {
  ep::BlockNormArgs a{};
  a.T = n->num_tokens;
  a.H = n->hidden;
  a.eps = n->eps;
  a.scale = n->residual_scale;
  a.weight32 = n->weight_type == EP_REAL_FP32;
  a.gate_per_token = n->gate && n->gate_per_token;
  a.post = n->post_weight;
  a.pre = n->pre_weight;
  a.gate = n->gate;
  a.mask = n->token_mask;
  return a;
}

ep::GateArgs gate_args(const void* logits, ep_logits_t type, int64_t ld, const uint8_t* mask, int T, int E, int k,
                       ep_gate_score_t score, float coef, int bits) {
  ep::GateArgs p{};
  p.logits = logits;
  p.ld = ld;
  p.mask = mask;
  p.T = T;
  p.E = E;
  p.k = k;
  p.groups = p.keep = 1;
  p.sigmoid = score == EP_GATE_SIGMOID;
  p.ids32 = bits == 32;
  p.coef = coef;
  p.vec = words16(logits, type, ld, E);
  return p;
}

}  // namespace

extern "C" {

ep_status_t ep_gate_workspace_bytes(int num_experts, int64_t* bytes) {
  if (num_experts < 1 || num_experts > 4096 || !bytes) return EP_ERR_INVALID_ARG;
  *bytes = static_cast<int64_t>(ep::gate_work_bytes(num_experts));
  return EP_OK;
}

ep_status_t ep_gate_forward(const void* logits, ep_logits_t logits_type, int64_t logits_ld, const uint8_t* token_mask,
                            int T, int E, int k, int num_groups, int topk_groups, ep_gate_score_t score,
                            float loss_coef, void* topk_idx, int topk_idx_bits, float* topk_weights,
                            int* expert_count, float* expert_prob, float* loss, void* workspace, int num_sms,
                            ep_stream_t stream) {
  if (!gate_ok(logits, logits_type, logits_ld, T, E, k, score)) return EP_ERR_INVALID_ARG;
  if (num_groups < 1 || num_groups > 64 || E % num_groups != 0 || topk_groups < 1 || topk_groups > num_groups)
    return EP_ERR_INVALID_ARG;
  if ((topk_idx_bits != 32 && topk_idx_bits != 64) || !expert_count || !expert_prob || !loss || !workspace ||
      (T > 0 && (!topk_idx || !topk_weights)))
    return EP_ERR_INVALID_ARG;
  if (!aligned(topk_idx, topk_idx_bits / 8) || !aligned(topk_weights, 4) || !aligned(expert_count, 4) ||
      !aligned(expert_prob, 4) || !aligned(loss, 4) || !aligned(workspace, 16))
    return EP_ERR_INVALID_ARG;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::GateArgs p = gate_args(logits, logits_type, logits_ld, token_mask, T, E, k, score, loss_coef, topk_idx_bits);
  p.groups = num_groups;
  p.keep = topk_groups;
  p.idx = topk_idx;
  p.weights = topk_weights;
  p.count = expert_count;
  p.prob = expert_prob;
  p.loss = loss;
  p.work = static_cast<unsigned*>(workspace);
  int log2_T = 0;
  while ((1LL << log2_T) < T) ++log2_T;
  p.fixed = static_cast<float>(1ull << (63 - log2_T));
  return status_of(ep::launch_gate(p, logits_type == EP_LOGITS_BF16, false, sms, reinterpret_cast<cudaStream_t>(stream)),
                   "ep_gate_forward launch");
}

ep_status_t ep_gate_backward(const void* logits, ep_logits_t logits_type, int64_t logits_ld,
                             const uint8_t* token_mask, int T, int E, int k, ep_gate_score_t score, float loss_coef,
                             const void* topk_idx, int topk_idx_bits, const int* expert_count,
                             const float* grad_topk_weights, const float* grad_loss, void* grad_logits,
                             int64_t grad_logits_ld, int num_sms, ep_stream_t stream) {
  if (!gate_ok(logits, logits_type, logits_ld, T, E, k, score)) return EP_ERR_INVALID_ARG;
  if ((topk_idx_bits != 32 && topk_idx_bits != 64) || !expert_count || grad_logits_ld < E ||
      (T > 0 && (!topk_idx || !grad_logits)))
    return EP_ERR_INVALID_ARG;
  if (!aligned(topk_idx, topk_idx_bits / 8) || !aligned(expert_count, 4) || !aligned(grad_topk_weights, 4) ||
      !aligned(grad_loss, 4) || !aligned(grad_logits, logits_type == EP_LOGITS_FP32 ? 4 : 2))
    return EP_ERR_INVALID_ARG;
  if (T == 0) return EP_OK;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::GateArgs p = gate_args(logits, logits_type, logits_ld, token_mask, T, E, k, score, loss_coef, topk_idx_bits);
  p.idx = const_cast<void*>(topk_idx);
  p.count = const_cast<int*>(expert_count);
  p.grad_weights = grad_topk_weights;
  p.grad_loss = grad_loss;
  p.grad_logits = grad_logits;
  p.grad_ld = grad_logits_ld;
  p.grad_vec = words16(grad_logits, logits_type, grad_logits_ld, E);
  return status_of(ep::launch_gate(p, logits_type == EP_LOGITS_BF16, true, sms, reinterpret_cast<cudaStream_t>(stream)),
                   "ep_gate_backward launch");
}

ep_status_t ep_grouped_matmul(const ep_groups_t* groups, const ep_fp8_rows_t* x, const void* w, const float* w_scales,
                              int N, int K, void* out, int num_sms, ep_stream_t stream) {
  if (!groups_ok(groups) || N < 8 || N % 8 != 0 || K < 128 || K % 128 != 0) return EP_ERR_INVALID_ARG;
  if (static_cast<long long>(groups->num_groups) * N > INT_MAX || !tiles_ok(groups, N) || !w || !w_scales ||
      !aligned(w, 16) || !aligned(w_scales, 4))
    return EP_ERR_INVALID_ARG;
  if (groups->rows == 0) return EP_OK;
  if (!rows_ok(x) || !out || !aligned(out, 16)) return EP_ERR_INVALID_ARG;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::MatmulArgs p{};
  p.groups = groups_of(groups);
  p.x = rows_of(x);
  p.w = w;
  p.w_scales = w_scales;
  p.N = N;
  p.K = K;
  p.out = static_cast<uint16_t*>(out);
  return status_of(ep::launch_grouped_matmul(p, sms, reinterpret_cast<cudaStream_t>(stream)), "ep_grouped_matmul launch");
}

ep_status_t ep_grouped_matmul_swiglu(const ep_groups_t* groups, const ep_fp8_rows_t* x, const void* w,
                                     const float* w_scales, int F, int K, const float* row_weights,
                                     const ep_fp8_rows_t* act, const ep_fp8_rows_t* pre, int num_sms,
                                     ep_stream_t stream) {
  if (!groups_ok(groups) || F < 128 || F % 128 != 0 || K < 128 || K % 128 != 0) return EP_ERR_INVALID_ARG;
  if (static_cast<long long>(groups->num_groups) * F * 2 > INT_MAX || !tiles_ok(groups, 2 * F) || !w || !w_scales || !aligned(w, 16) ||
      !aligned(w_scales, 4) || !aligned(row_weights, 4))
    return EP_ERR_INVALID_ARG;
  if (groups->rows == 0) return EP_OK;
  if (!rows_ok(x) || !rows_ok(act) || (pre && !rows_ok(pre))) return EP_ERR_INVALID_ARG;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::MatmulArgs p{};
  p.groups = groups_of(groups);
  p.x = rows_of(x);
  p.w = w;
  p.w_scales = w_scales;
  p.N = 2 * F;
  p.K = K;
  p.act = rows_of(act);
  if (pre) p.pre = rows_of(pre);
  p.row_weights = row_weights;
  return status_of(ep::launch_grouped_matmul(p, sms, reinterpret_cast<cudaStream_t>(stream)),
                   "ep_grouped_matmul_swiglu launch");
}

static bool w4_ok(const ep_groups_t* g, const void* w, const void* w_scales, int N, int K) {
  return groups_ok(g) && K >= 128 && K % 128 == 0 && static_cast<long long>(g->num_groups) * N <= INT_MAX &&
         (g->rows / ep::kTile4Rows + g->num_groups + 1) * ((N + 127) / 128) < INT_MAX / 2 && w && w_scales &&
         aligned(w, 32) && aligned(w_scales, 16);
}

ep_status_t ep_grouped_matmul_w4(const ep_groups_t* groups, const ep_fp8_rows_t* x, const void* w,
                                 const uint8_t* w_scales, int N, int K, void* out, int num_sms, ep_stream_t stream) {
  if (N < 8 || N % 8 != 0 || !w4_ok(groups, w, w_scales, N, K)) return EP_ERR_INVALID_ARG;
  if (groups->rows == 0) return EP_OK;
  if (!rows_ok(x) || !out || !aligned(out, 16)) return EP_ERR_INVALID_ARG;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::Matmul4Args p{};
  p.groups = groups_of(groups);
  p.x = rows_of(x);
  p.w = w;
  p.w_scales = w_scales;
  p.N = N;
  p.K = K;
  p.out = static_cast<uint16_t*>(out);
  return status_of(ep::launch_grouped_matmul_w4(p, sms, reinterpret_cast<cudaStream_t>(stream)),
                   "ep_grouped_matmul_w4 launch");
}

ep_status_t ep_grouped_matmul_w4_swiglu(const ep_groups_t* groups, const ep_fp8_rows_t* x, const void* w,
                                        const uint8_t* w_scales, int F, int K, const float* row_weights,
                                        const ep_fp8_rows_t* act, int num_sms, ep_stream_t stream) {
  if (F < 128 || F % 128 != 0 || F > INT_MAX / 2 || !w4_ok(groups, w, w_scales, 2 * F, K) || !aligned(row_weights, 4))
    return EP_ERR_INVALID_ARG;
  if (groups->rows == 0) return EP_OK;
  if (!rows_ok(x) || !rows_ok(act)) return EP_ERR_INVALID_ARG;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::Matmul4Args p{};
  p.groups = groups_of(groups);
  p.x = rows_of(x);
  p.w = w;
  p.w_scales = w_scales;
  p.N = 2 * F;
  p.K = K;
  p.act = rows_of(act);
  p.row_weights = row_weights;
  return status_of(ep::launch_grouped_matmul_w4(p, sms, reinterpret_cast<cudaStream_t>(stream)),
                   "ep_grouped_matmul_w4_swiglu launch");
}

ep_status_t ep_grouped_swiglu_backward(const ep_groups_t* groups, const void* grad_act, const ep_fp8_rows_t* pre,
                                       const float* row_weights, int F, const ep_fp8_rows_t* grad_pre,
                                       float* grad_row_weights, int num_sms, ep_stream_t stream) {
  if (!groups_ok(groups) || F < 128 || F % 128 != 0 || F > INT_MAX / 2) return EP_ERR_INVALID_ARG;
  if (!aligned(row_weights, 4) || !aligned(grad_row_weights, 4)) return EP_ERR_INVALID_ARG;
  if (groups->rows == 0) return EP_OK;
  if (!grad_act || !aligned(grad_act, 16) || !rows_ok(pre) || !rows_ok(grad_pre)) return EP_ERR_INVALID_ARG;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::SwigluBackwardArgs p{};
  p.groups = groups_of(groups);
  p.grad_act = static_cast<const uint16_t*>(grad_act);
  p.pre = rows_of(pre);
  p.row_weights = row_weights;
  p.grad_pre = rows_of(grad_pre);
  p.grad_row_weights = grad_row_weights;
  p.F = F;
  return status_of(ep::launch_swiglu_backward(p, sms, reinterpret_cast<cudaStream_t>(stream)),
                   "ep_grouped_swiglu_backward launch");
}

ep_status_t ep_grouped_weight_grad(const ep_groups_t* groups, const ep_fp8_rows_t* grad_out, int N,
                                   const ep_fp8_rows_t* x, int K, void* grad_w, int num_sms, ep_stream_t stream) {
  if (!groups_ok(groups) || N < 128 || N % 128 != 0 || K < 128 || K % 128 != 0) return EP_ERR_INVALID_ARG;
  if (static_cast<long long>(groups->num_groups) * (N / 128) * ((K + 255) / 256) > INT_MAX / 2 ||
      static_cast<long long>(groups->num_groups) * N > INT_MAX || !grad_w || !aligned(grad_w, 16))
    return EP_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (groups->rows == 0)
    return status_of(cudaMemsetAsync(grad_w, 0, static_cast<size_t>(groups->num_groups) * N * K * 2, s), "weight gradient memset");
  if (!rows_ok(grad_out) || !rows_ok(x)) return EP_ERR_INVALID_ARG;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::WeightGradArgs p{};
  p.groups = groups_of(groups);
  p.dy = rows_of(grad_out);
  p.x = rows_of(x);
  p.N = N;
  p.K = K;
  p.dw = static_cast<uint16_t*>(grad_w);
  return status_of(ep::launch_weight_grad(p, sms, s), "ep_grouped_weight_grad launch");
}

ep_status_t ep_block_norm_forward(const ep_block_norm_t* norm, const void* residual, const void* y, void* new_residual,
                                  void* x, float* rstd, int num_sms, ep_stream_t stream) {
  if (!norm_ok(norm)) return EP_ERR_INVALID_ARG;
  const bool any = norm->num_tokens > 0;  // tensors without tokens have no address
  if ((norm->pre_weight && any && !x) || (!norm->pre_weight && x)) return EP_ERR_INVALID_ARG;
  if (any && (!residual || (y ? !new_residual : norm->post_weight || norm->gate || !x))) return EP_ERR_INVALID_ARG;
  if (!aligned(residual, 16) || !aligned(y, 16) || !aligned(new_residual, 16) || !aligned(x, 16) || !aligned(rstd, 4))
    return EP_ERR_INVALID_ARG;
  if (!any) return EP_OK;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::BlockNormArgs a = norm_args(norm);
  a.residual = residual;
  a.y = y;
  a.new_residual = new_residual;
  a.x = x;
  a.rstd = rstd;
  return status_of(ep::launch_block_norm(a, norm->residual_type == EP_REAL_FP32, sms, reinterpret_cast<cudaStream_t>(stream)),
                   "ep_block_norm_forward launch");
}

ep_status_t ep_block_norm_workspace_bytes(int hidden, int64_t* bytes) {
  if (hidden < 8 || hidden % 8 != 0 || hidden > ep::kBlockNormMaxHidden || !bytes) return EP_ERR_INVALID_ARG;
  *bytes = static_cast<int64_t>(ep::kBlockNormMaxBlocks) * 2 * sizeof(float) * hidden;
  return EP_OK;
}

ep_status_t ep_block_norm_backward(const ep_block_norm_t* norm, const void* new_residual, const void* y,
                                   const float* rstd, const void* grad_new_residual, const void* grad_x,
                                   void* grad_residual, void* grad_y, void* grad_gate, float* grad_post_weight,
                                   float* grad_pre_weight, void* workspace, int num_sms, ep_stream_t stream) {
  if (!norm_ok(norm)) return EP_ERR_INVALID_ARG;
  const bool any = norm->num_tokens > 0;
  const bool per_token = norm->gate && norm->gate_per_token;
  if ((grad_gate && !norm->gate) || (grad_post_weight && !norm->post_weight) ||
      (grad_pre_weight && (!norm->pre_weight || (any && !grad_x))) || (grad_x && !norm->pre_weight))
    return EP_ERR_INVALID_ARG;
  const bool block = grad_y || grad_gate || grad_post_weight;
  if (any && ((grad_x && (!new_residual || !rstd)) || (block && norm->post_weight && (!y || !rstd)) || (grad_gate && !y)))
    return EP_ERR_INVALID_ARG;
  const bool sums = grad_pre_weight || grad_post_weight || (grad_gate && !per_token);
  if (sums && any && !workspace) return EP_ERR_INVALID_ARG;
  for (const void* p : {new_residual, y, grad_new_residual, grad_x, static_cast<const void*>(grad_residual),
                        static_cast<const void*>(grad_y), static_cast<const void*>(grad_gate),
                        static_cast<const void*>(grad_post_weight), static_cast<const void*>(grad_pre_weight),
                        static_cast<const void*>(workspace)})
    if (!aligned(p, 16)) return EP_ERR_INVALID_ARG;
  if (!aligned(rstd, 4)) return EP_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!any) {
    cudaError_t e = cudaSuccess;
    for (float* p : {grad_pre_weight, grad_post_weight, per_token ? nullptr : static_cast<float*>(grad_gate)})
      if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, sizeof(float) * norm->hidden, s);
    return status_of(e, "ep_block_norm_backward memset");
  }
  if (!block && !grad_residual && !grad_pre_weight) return EP_OK;
  int sms = 0;
  ep_status_t st = sm_count(num_sms, &sms);
  if (st != EP_OK) return st;
  ep::BlockNormBackwardArgs a{};
  a.n = norm_args(norm);
  a.n.new_residual = const_cast<void*>(new_residual);
  a.n.y = y;
  a.n.rstd = const_cast<float*>(rstd);
  a.grad_new = grad_new_residual;
  a.grad_x = grad_x;
  a.grad_residual = grad_residual;
  a.grad_y = grad_y;
  a.grad_gate = grad_gate;
  a.grad_post = grad_post_weight;
  a.grad_pre = grad_pre_weight;
  a.partial = static_cast<float*>(workspace);
  return status_of(ep::launch_block_norm_backward(a, norm->residual_type == EP_REAL_FP32, sms, s),
                   "ep_block_norm_backward launch");
}

}  // extern "C"
