// few_api.cu -- the C ABI's few-token layers (include/moe_prefill.h): argument checks and launches.

#include <cuda_runtime.h>

#include "few.h"
#include "internal.h"

using namespace moe;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool sizes_ok(const moe_prefill_config* c, int shared_inter, int fp8, int T) {
  if (c == nullptr || T < 1 || T > MOE_FEW_MAX_TOKENS) return false;
  const int piece = fp8 ? 128 : 256;
  return c->hidden >= piece && c->hidden % piece == 0 && c->hidden <= (1 << 20) && c->moe_intermediate >= piece &&
         c->moe_intermediate % piece == 0 && c->moe_intermediate <= (1 << 20) && c->num_experts >= 1 &&
         c->num_experts <= MOE_FEW_MAX_EXPERTS && c->top_k >= 1 && c->top_k <= 32 && c->top_k <= c->num_experts &&
         shared_inter >= 0 && shared_inter % 128 == 0 && shared_inter <= (1 << 20) && (fp8 || shared_inter == 0);
}

// What both formats' calls have in common.
int common(const moe_prefill_config* c, const uint16_t* x, int T, const uint16_t* w_router, const float* logits,
           const float* bias, int shared_inter, int fp8, const void* ws, size_t ws_bytes, uint16_t* out, FewArgs& a,
           FewLayout& l) {
  if (c == nullptr || (w_router == nullptr) == (logits == nullptr) || (w_router != nullptr && x == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!(c->swiglu_limit > 0.f) || (c->flags & ~MOE_FWD_NO_MULTICAST) != 0) return MOE_ERR_INVALID_ARG;
  if (!sizes_ok(c, shared_inter, fp8, T)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (ws == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(logits, 4) || !aligned(bias, 4) || !aligned(ws, 256) ||
      !aligned(out, 2))
    return MOE_ERR_INVALID_ARG;
  a.x = x;
  a.w_router = w_router;
  a.logits = logits;
  a.bias = bias;
  a.T = T;
  a.H = c->hidden;
  a.I = c->moe_intermediate;
  a.Is = shared_inter;
  a.E = c->num_experts;
  a.k = c->top_k;
  a.first = 0;
  a.count = a.E;
  a.renormalize = c->renormalize;
  a.routed_scale = c->routed_scale;
  a.limit = c->swiglu_limit;
  a.out = out;
  a.wait_ns = gemm_wait_limit_ns();
  l = fp8 ? few_fp8_layout(T, a.H, a.I, a.Is, a.E, a.k) : few_w4_layout(T, a.H, a.I, a.Is, a.E, a.k);
  return ws_bytes < l.total ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

// A weight [count][N, K] of exactly these sizes.
int weight_ok(const moe_fp8_weight* w, int N, int K) {
  if (w == nullptr || w->q == nullptr || w->s == nullptr) return MOE_ERR_INVALID_ARG;
  if (w->N != N || w->K != K || w->count < 1 || w->first < 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(w->q, 16) || !aligned(w->s, 4) || w->ld < K || w->ld % 16 != 0 || w->ld >= (1ll << 40))
    return MOE_ERR_INVALID_ARG;
  if (w->count > 1 && (w->expert_stride % 16 != 0 || w->expert_stride < w->ld * (N - 1) + K ||
                       w->expert_stride >= (1ll << 40)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

FewFp8Weight view(const moe_fp8_weight* w) { return FewFp8Weight{w->q, w->ld, w->count > 1 ? w->expert_stride : 0, w->s}; }

}  // namespace

extern "C" {

size_t moe_few_workspace_bytes(const moe_prefill_config* cfg, int fp8, int shared_intermediate, int T) {
  if (!sizes_ok(cfg, shared_intermediate, fp8, T)) return 0;
  const int E = cfg->num_experts, k = cfg->top_k, H = cfg->hidden, I = cfg->moe_intermediate;
  return (fp8 ? few_fp8_layout(T, H, I, shared_intermediate, E, k) : few_w4_layout(T, H, I, shared_intermediate, E, k)).total;
}

int moe_fp8_few_forward(const moe_prefill_config* cfg, const uint16_t* x, const moe_fp8_rows* rows, int T,
                        const uint16_t* w_router, const float* logits, const float* router_bias,
                        const moe_fp8_weight* gate_up, const moe_fp8_weight* down, const moe_fp8_weight* shared_gate_up,
                        const moe_fp8_weight* shared_down, float shared_limit, void* ws, size_t ws_bytes, uint16_t* out,
                        void* stream) {
  if ((shared_gate_up == nullptr) != (shared_down == nullptr) || (x == nullptr && rows == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (shared_down != nullptr && (shared_down->K < 1 || !(shared_limit > 0.f))) return MOE_ERR_INVALID_ARG;
  FewArgs a = {};
  FewLayout l;
  int rc = common(cfg, x, T, w_router, logits, router_bias, shared_down != nullptr ? shared_down->K : 0, 1, ws, ws_bytes,
                  out, a, l);
  if (rc != MOE_OK) return rc;
  if ((rc = weight_ok(gate_up, 2 * a.I, a.H)) != MOE_OK || (rc = weight_ok(down, a.H, a.I)) != MOE_OK) return rc;
  if (gate_up->first != down->first || gate_up->count != down->count || gate_up->count > a.E - gate_up->first)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (shared_down != nullptr) {
    if ((rc = weight_ok(shared_gate_up, 2 * a.Is, a.H)) != MOE_OK || (rc = weight_ok(shared_down, a.H, a.Is)) != MOE_OK)
      return rc;
    if (gate_up->first != 0) return MOE_ERR_UNSUPPORTED_SHAPE;  // (the shared expert goes with expert 0)
    a.w8s[0] = view(shared_gate_up);
    a.w8s[1] = view(shared_down);
    a.shared_limit = shared_limit;
  }
  if (rows != nullptr) {
    if (rows->q == nullptr || rows->s == nullptr || !aligned(rows->q, 16) || !aligned(rows->s, 4) || rows->ld < a.H ||
        rows->ld % 16 != 0)
      return MOE_ERR_INVALID_ARG;
    if (rows->rows != T) return MOE_ERR_UNSUPPORTED_SHAPE;
    a.rows_q = rows->q;
    a.rows_ld = rows->ld;
    a.rows_s = rows->s;
    a.rows_s_row = rows->s_row;
    a.rows_s_grp = rows->s_grp;
  }
  a.first = gate_up->first;
  a.count = gate_up->count;
  a.w8[0] = view(gate_up);
  a.w8[1] = view(down);
  if ((rc = ensure_device()) != MOE_OK) return rc;
  a.err = device_error_word();
  return few_fp8_launch(a, l, ws, static_cast<cudaStream_t>(stream));
}

int moe_w4a16_few_forward(const moe_prefill_config* cfg, const uint16_t* x, int T, const uint16_t* w_router,
                          const float* logits, const float* router_bias, const moe_expert_table* w_gate_up,
                          const moe_expert_table* w_down, const uint16_t* shared_out, void* ws, size_t ws_bytes,
                          uint16_t* out, void* stream) {
  if (x == nullptr || w_gate_up == nullptr || w_down == nullptr || !aligned(shared_out, 2)) return MOE_ERR_INVALID_ARG;
  FewArgs a = {};
  FewLayout l;
  int rc = common(cfg, x, T, w_router, logits, router_bias, 0, 0, ws, ws_bytes, out, a, l);
  if (rc != MOE_OK) return rc;
  const ExpertTableView gu = expert_table_view(w_gate_up), dn = expert_table_view(w_down);
  if (gu.E != a.E || gu.N != 2 * a.I || gu.K != a.H || dn.E != a.E || dn.N != a.H || dn.K != a.I)
    return MOE_ERR_INVALID_ARG;
  if ((rc = ensure_device()) != MOE_OK) return rc;
  if (current_device_index() != gu.device || current_device_index() != dn.device) return MOE_ERR_INVALID_ARG;
  a.w4[0] = FewW4Weight{gu.maps, gu.packed, gu.scales, gu.scale2};
  a.w4[1] = FewW4Weight{dn.maps, dn.packed, dn.scales, dn.scale2};
  a.shared_out = shared_out;
  a.err = device_error_word();
  return few_w4_launch(a, l, ws, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
