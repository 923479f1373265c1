// fp8_api.cu -- the C ABI's FP8 calls (include/moe_prefill.h): argument checks and launches.

#include <cuda_runtime.h>

#include "internal.h"

using namespace moe;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
bool dtype_ok(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }

// Rows of one TMA operand: codes 16-byte aligned, rows a multiple of 16 bytes apart (below 2^40 bytes).
bool codes_ok(const uint8_t* q, int64_t ld, int K) { return aligned(q, 16) && ld >= K && ld % 16 == 0 && ld < (1ll << 40); }

int check(const moe_fp8_rows* A, const moe_fp8_weight* W, int R, int E) {
  if (A == nullptr || W == nullptr || A->q == nullptr || A->s == nullptr || W->q == nullptr || W->s == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (W->N < 1 || W->K < 1 || W->count < 1 || W->first < 0 || E < 1 || E > MOE_FP8_MAX_EXPERTS ||
      W->count > E - W->first || R < 0 || A->rows < 0)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (R > 0 && A->rows < 1) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(A->s, 4) || !aligned(W->s, 4)) return MOE_ERR_INVALID_ARG;
  if (!codes_ok(A->q, A->ld, W->K) || !codes_ok(W->q, W->ld, W->K)) return MOE_ERR_INVALID_ARG;
  // (the experts' stride is a TMA stride too; a single expert's is not used)
  if (W->count > 1 && (W->expert_stride % 16 != 0 || W->expert_stride < W->ld * (W->N - 1) + W->K ||
                       W->expert_stride >= (1ll << 40)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

Fp8Gemm make(const moe_fp8_rows* A, const int32_t* gather_ids, const moe_fp8_weight* W, const int32_t* offsets, int E,
             int R) {
  Fp8Gemm d = {};
  d.W = W->q;
  d.ldw = W->ld;
  d.w_expert = W->count > 1 ? W->expert_stride : (W->ld * (int64_t)W->N);
  Fp8GemmArgs& a = d.args;
  a.A = A->q;
  a.lda = A->ld;
  a.sa = A->s;
  a.sa_row = A->s_row;
  a.sa_grp = A->s_grp;
  a.sw = W->s;
  a.gather = gather_ids;
  a.offsets = offsets;
  a.wait_ns = gemm_wait_limit_ns();
  a.err = device_error_word();
  a.E = E;
  a.e_first = W->first;
  a.e_count = W->count;
  a.N = W->N;
  a.K = W->K;
  a.R = R;
  a.a_rows = A->rows;
  a.nblk = (W->N + 127) / 128;
  return d;
}

int product(const moe_fp8_rows* A, const int32_t* gather_ids, const moe_fp8_weight* W, const int32_t* offsets, int E,
            int R, void* C, int64_t ldc, int c_dtype, void* stream) {
  int rc = check(A, W, R, E);
  if (rc != MOE_OK) return rc;
  if (C == nullptr || !dtype_ok(c_dtype)) return MOE_ERR_INVALID_ARG;
  if (ldc < W->N || ldc % 8 != 0 || ldc >= (1ll << 38)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(C, 16)) return MOE_ERR_INVALID_ARG;
  if (gather_ids == nullptr && A->rows < R) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((rc = ensure_device()) != MOE_OK || R == 0) return rc;
  Fp8Gemm d = make(A, gather_ids, W, offsets, E, R);
  d.args.C = C;
  d.args.ldc = ldc;
  d.args.c_dtype = c_dtype;
  return fp8_gemm_launch(d, as_stream(stream));
}

}  // namespace

extern "C" {

int moe_fp8_quantize_rows(const void* x, int x_dtype, int64_t ld_x, int R, int K, uint8_t* q, int64_t ld_q, float* s,
                          int64_t s_row, int64_t s_grp, void* stream) {
  if (x == nullptr || q == nullptr || s == nullptr || !dtype_ok(x_dtype)) return MOE_ERR_INVALID_ARG;
  if (R < 0 || K < 1 || ld_x < K) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!codes_ok(q, ld_q, K) || !aligned(s, 4) || !aligned(x, x_dtype == MOE_DTYPE_BF16 ? 2 : 4))
    return MOE_ERR_INVALID_ARG;
  const int rc = ensure_device();
  if (rc != MOE_OK || R == 0) return rc;
  return fp8_quantize_rows_launch(x, x_dtype, ld_x, R, K, q, ld_q, s, s_row, s_grp, as_stream(stream));
}

int moe_fp8_quantize_blocks(const void* w, int w_dtype, int64_t ld_w, int N, int K, uint8_t* q, int64_t ld_q, float* s,
                            void* stream) {
  if (w == nullptr || q == nullptr || s == nullptr || !dtype_ok(w_dtype)) return MOE_ERR_INVALID_ARG;
  if (N < 1 || N > 65535 * 128 || K < 1 || ld_w < K) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!codes_ok(q, ld_q, K) || !aligned(s, 4) || !aligned(w, w_dtype == MOE_DTYPE_BF16 ? 2 : 4))
    return MOE_ERR_INVALID_ARG;
  const int rc = ensure_device();
  if (rc != MOE_OK) return rc;
  return fp8_quantize_blocks_launch(w, w_dtype, ld_w, N, K, q, ld_q, s, as_stream(stream));
}

int moe_fp8_gemm(const moe_fp8_rows* A, const moe_fp8_weight* W, void* C, int64_t ldc, int c_dtype, void* stream) {
  if (A == nullptr || W == nullptr) return MOE_ERR_INVALID_ARG;
  if (W->first != 0 || W->count != 1) return MOE_ERR_UNSUPPORTED_SHAPE;
  return product(A, nullptr, W, nullptr, 1, A->rows, C, ldc, c_dtype, stream);
}

int moe_fp8_grouped_gemm(const moe_fp8_rows* A, const int32_t* gather_ids, const moe_fp8_weight* W,
                         const int32_t* expert_offsets, int E, int R, void* C, int64_t ldc, int c_dtype, void* stream) {
  if (expert_offsets == nullptr) return MOE_ERR_INVALID_ARG;
  return product(A, gather_ids, W, expert_offsets, E, R, C, ldc, c_dtype, stream);
}

int moe_fp8_grouped_gemm_swiglu(const moe_fp8_rows* A, const int32_t* gather_ids, const moe_fp8_weight* W,
                                const int32_t* expert_offsets, int E, int R, float limit, uint8_t* act, int64_t ld_act,
                                float* act_s, int64_t act_s_row, int64_t act_s_grp, void* stream) {
  if (expert_offsets == nullptr) return MOE_ERR_INVALID_ARG;
  int rc = check(A, W, R, E);
  if (rc != MOE_OK) return rc;
  if (act == nullptr || act_s == nullptr || !(limit > 0.f)) return MOE_ERR_INVALID_ARG;
  if (W->N % 256 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!codes_ok(act, ld_act, W->N / 2) || !aligned(act_s, 4)) return MOE_ERR_INVALID_ARG;
  if (gather_ids == nullptr && A->rows < R) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((rc = ensure_device()) != MOE_OK || R == 0) return rc;
  Fp8Gemm d = make(A, gather_ids, W, expert_offsets, E, R);
  Fp8GemmArgs& a = d.args;
  a.half = W->N / 2;
  a.limit = limit;
  a.q = act;
  a.ld_q = ld_act;
  a.s = act_s;
  a.s_row = act_s_row;
  a.s_grp = act_s_grp;
  return fp8_gemm_launch(d, as_stream(stream));
}

}  // extern "C"
