// rms_norm.cu -- the step in front of the experts: residual addition, root-mean-square norm, and the row
// quantiser on its result, in one pass over the row.
//
//   h = x + r,   y = h / sqrt(mean(h^2) + eps) * w,   (q, s) = codes and scales of y, 128 columns to a scale
//
// in FP32 from the elements to the outputs: h is rounded to the residual's type where it is stored, but y is
// made of the unrounded sum, and the codes are made of the unrounded y (fp8_quant.cu has the quantiser).
// The squares are summed in FP32 in a fixed order: by thread, by shuffles, by warps.
//
// A row belongs to one CTA, which holds it in registers between the sum of squares and the outputs, so every
// element is read once and written once; the CTAs that an SM holds beside each other (6 of 320 threads at 5120
// columns) hide the two barriers.  Two layouts:
//   VEC  16 consecutive columns to a thread, 8 threads to a group of 128, 16-byte loads and stores; for
//        operands whose rows all start on 16-byte boundaries
//   any  4 columns to a thread, 32 apart, a warp to a group: element loads and stores that still coalesce
//
// Bound by memory.

#include <algorithm>

#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace rn {

constexpr int G = 128;

MOE_DEV float load1(const void* p, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16)
              : reinterpret_cast<const float*>(p)[i];
}
MOE_DEV void store1(void* p, int64_t i, float v, bool bf16) {
  if (bf16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<float*>(p)[i] = v;
}

// n <= 16 consecutive elements from i on; the wide form for n = 16 on 16-byte boundaries
MOE_DEV void load16(const void* p, int64_t i, bool bf16, int n, float (&v)[16]) {
  if (n == 16 && bf16) {
    const uint4* a = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
    const uint4 lo = a[0], hi = a[1];
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[2 * j] = bf16_lo(w[j]);
      v[2 * j + 1] = bf16_hi(w[j]);
    }
  } else if (n == 16) {
    const float4* a = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 f = a[j];
      v[4 * j] = f.x;
      v[4 * j + 1] = f.y;
      v[4 * j + 2] = f.z;
      v[4 * j + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = j < n ? load1(p, i + j, bf16) : 0.f;
  }
}
MOE_DEV void store16(void* p, int64_t i, bool bf16, int n, const float (&v)[16]) {
  if (n == 16 && bf16) {
    uint4* a = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      a[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                        pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
  } else if (n == 16) {
    float4* a = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < n) store1(p, i + j, v[j], bf16);
  }
}

// Sum over the row's threads: the warp's by shuffles, then over the row's warps in their order.
MOE_DEV float row_sum(float v, float* s_part, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_part[0];
  for (int i = 1; i < warps; ++i) v += s_part[i];
  return v;
}

// A CTA to a row, or (rows of one warp) a warp to a row.  C: pieces of a row to a thread, 16 columns each (VEC)
// or 4 (any).
template <int C, bool VEC>
__global__ void __launch_bounds__(512) norm_kernel(RmsNormArgs a, int warps) {
  constexpr int N = VEC ? 16 : 4;
  __shared__ float s_part[32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_cta = warps == 1 ? (int)(blockDim.x >> 5) : 1;
  const int row = blockIdx.x * per_cta + (warps == 1 ? warp : 0);
  if (row >= a.R) return;  // (whole warps, and only where no barrier follows)
  const int tid = warps == 1 ? lane : (int)threadIdx.x, threads = warps * 32;
  const int64_t xr = (int64_t)row * a.ld_x, rr = (int64_t)row * a.ld_r;
  float h[C][N];
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (VEC) {
      const int k0 = (c * threads + tid) * 16, n = max(0, min(16, a.K - k0));
      load16(a.x, xr + k0, a.x_bf16, n, h[c]);
      if (a.r != nullptr) {
        float r[16];
        load16(a.r, rr + k0, a.r_bf16, n, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) h[c][i] += r[i];
      }
    } else {
      const int k0 = (c * warps + (warps == 1 ? 0 : warp)) * G + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 32 * i;
        h[c][i] = k < a.K ? load1(a.x, xr + k, a.x_bf16) : 0.f;
        if (a.r != nullptr && k < a.K) h[c][i] += load1(a.r, rr + k, a.r_bf16);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) sum = __fmaf_rn(h[c][i], h[c][i], sum);
  }
  sum = row_sum(sum, s_part, warps);
  const float inv = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)a.K) + a.eps));
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (VEC) {
      const int k0 = (c * threads + tid) * 16, n = max(0, min(16, a.K - k0));
      if (a.r != nullptr) store16(a.h, (int64_t)row * a.ld_h + k0, a.r_bf16, n, h[c]);
      float w[16];
      load16(a.w, k0, a.w_bf16, n, w);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        h[c][i] = h[c][i] * inv * w[i];
        if (i < n) m = max(m, __float_as_uint(h[c][i]) & 0x7FFFFFFFu);
      }
      if (a.y != nullptr) store16(a.y, (int64_t)row * a.ld_y + k0, true, n, h[c]);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      float scale, by;
      fp8_scale(m, scale, by);
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[i] = pack_e4m3x4(h[c][4 * i] * by, h[c][4 * i + 1] * by, h[c][4 * i + 2] * by, h[c][4 * i + 3] * by);
      uint8_t* dst = a.q + (int64_t)row * a.ld_q + k0;
      if (n == 16) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < n) dst[i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
      }
      if ((lane & 7) == 0 && k0 < a.K) a.s[row * a.s_row + (k0 / G) * a.s_grp] = scale;
    } else {
      const int grp = c * warps + (warps == 1 ? 0 : warp), k0 = grp * G + lane;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 32 * i;
        if (k >= a.K) continue;
        if (a.r != nullptr) store1(a.h, (int64_t)row * a.ld_h + k, h[c][i], a.r_bf16);
        h[c][i] = h[c][i] * inv * load1(a.w, k, a.w_bf16);
        if (a.y != nullptr) store1(a.y, (int64_t)row * a.ld_y + k, h[c][i], true);
        m = max(m, __float_as_uint(h[c][i]) & 0x7FFFFFFFu);
      }
      m = __reduce_max_sync(0xffffffffu, m);
      float scale, by;
      fp8_scale(m, scale, by);
      const uint32_t q = pack_e4m3x4(h[c][0] * by, h[c][1] * by, h[c][2] * by, h[c][3] * by);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k0 + 32 * i < a.K) a.q[(int64_t)row * a.ld_q + k0 + 32 * i] = (uint8_t)(q >> (8 * i));
      if (lane == 0 && grp * G < a.K) a.s[row * a.s_row + grp * a.s_grp] = scale;
    }
  }
}

bool wide(const void* p, int64_t ld, bool bf16) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (bf16 ? 2 : 4) % 16 == 0;
}

template <int C, bool VEC>
int launch(const RmsNormArgs& a, int warps, cudaStream_t st) {
  const int per_cta = warps == 1 ? 4 : 1;  // (rows of one warp: four to a CTA)
  const int grid = (a.R + per_cta - 1) / per_cta;
  return launch_pdl(norm_kernel<C, VEC>, dim3(grid), dim3(32 * warps * per_cta), 0, st, a, warps);
}

}  // namespace rn

int rms_norm_launch(const RmsNormArgs& a, cudaStream_t st) {
  using namespace rn;
  const bool vec = wide(a.x, a.ld_x, a.x_bf16) && wide(a.w, 0, a.w_bf16) &&
                   (a.r == nullptr || (wide(a.r, a.ld_r, a.r_bf16) && wide(a.h, a.ld_h, a.r_bf16))) &&
                   (a.y == nullptr || wide(a.y, a.ld_y, true));
  if (vec) {
    const int warps = (a.K + 511) / 512;  // of 16 columns a thread
    if (warps <= 16) return launch<1, true>(a, warps, st);
    if (warps <= 32) return launch<2, true>(a, (warps + 1) / 2, st);
    return launch<4, true>(a, (warps + 3) / 4, st);
  }
  const int groups = (a.K + G - 1) / G;
  if (groups <= 16) return launch<1, false>(a, groups, st);
  if (groups <= 64) return launch<4, false>(a, (groups + 3) / 4, st);
  return launch<16, false>(a, (groups + 15) / 16, st);
}

}  // namespace moe
