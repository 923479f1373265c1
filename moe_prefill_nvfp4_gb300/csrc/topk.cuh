// topk.cuh -- top-k routing of one row by one warp.
#pragma once

#include "common.cuh"

namespace moe {

// Order-preserving code of a selection key: a larger key gets a larger code, +0 and -0 the same
// one, and every key (-inf included) a code above 0, which marks "no candidate".
MOE_DEV uint32_t key_code(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u << 1) == 0u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One warp routes one row: top-k of (logit + bias) with ties to the lower expert index, weights
// from the unbiased logits (softmax over the k picks, or over all experts).  `lrow` may point to
// global or shared memory.  Shared by the standalone top-k kernel, the fused router + top-k
// kernel and the few-token layers.
template <int NPL>
MOE_DEV void topk_row(const float* lrow, const float* __restrict__ bias, int E, int k, int renormalize,
                      float routed_scale, int32_t* __restrict__ ids_row, float* __restrict__ wts_row, int* err) {
  const int lane = threadIdx.x & 31;
  float val[NPL], key[NPL];
  bool nan_seen = false;
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = lane + 32 * j;
    val[j] = e < E ? lrow[e] : -INFINITY;
    key[j] = e < E ? (bias ? val[j] + bias[e] : val[j]) : -INFINITY;
    if (e < E && (isnan(val[j]) || isnan(key[j]))) {
      nan_seen = true;
      key[j] = -INFINITY;
    }
  }
  if (__any_sync(0xffffffffu, nan_seen) && lane == 0) set_error(err, MOE_DEVERR_NAN_LOGIT);
  // selection s: the largest remaining key, ties to the lower expert.  A lane's candidate is its
  // best remaining code (strict >: the lower j, i.e. the lower expert, on ties); the warp takes
  // the largest code, then the lowest expert among the lanes holding it.
  uint32_t code[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) code[j] = lane + 32 * j < E ? key_code(key[j]) : 0u;
  int my_id = -1;
  for (int s = 0; s < k; ++s) {
    uint32_t bc = 0u, be = 0x7fffffffu;
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (code[j] > bc) {
        bc = code[j];
        be = lane + 32 * j;
      }
    const uint32_t mc = __reduce_max_sync(0xffffffffu, bc);
    const int pick = (int)__reduce_min_sync(0xffffffffu, bc == mc ? be : 0x7fffffffu);
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (pick == lane + 32 * j) code[j] = 0u;
    if (lane == s) my_id = pick;
  }
  // routing weights from the unbiased logits
  const bool mine = lane < k;
  const float l = mine ? lrow[my_id] : -INFINITY;
  float w;
  if (renormalize) {
    float m = l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ex = mine ? expf(l - m) : 0.f;
    float sum = ex;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = ex / sum;
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; ++j) m = fmaxf(m, val[j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (lane + 32 * j < E) sum += expf(val[j] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = mine ? expf(l - m) / sum : 0.f;
  }
  if (mine) {
    ids_row[lane] = my_id;
    wts_row[lane] = w * routed_scale;
  }
}

}  // namespace moe
