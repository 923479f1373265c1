// rms_norm.cu -- the step in front of the experts: residual addition, root-mean-square norm, and the row
// quantiser on its result, in one pass over the row.
//
//   h = x + r,   y = h / sqrt(mean(h^2) + eps) * w,   (q, s) = codes and scales of y, 128 columns to a scale
//
// in FP32 from the elements to the outputs: h is rounded to the residual's type where it is stored, but y is
// made of the unrounded sum.  The squares are summed in FP32 in a fixed order: by thread, by shuffles, by warps.
// A code is y / s rounded, and 1 / sqrt(...) is in both: it is h w * 448 / max |h w|, in pairs of FP32 numbers up to one
// rounding, since each rounding of a factor before it would be one more chance to end at the next code.
//
// Bound by memory.  A row belongs to one CTA, which holds it in registers between the sum of squares and the
// outputs, so every element is read once and written once.  Two layouts:
//   RING  8 threads to a group of 128, twice 8 consecutive columns each, 64 apart; a CTA goes through many rows, and while it
//         works on one, bulk copies bring the next into shared memory: some 100 KB of an SM on their way, with one barrier
//         to a row.  For operands whose rows all start on 16-byte boundaries.
//   any   4 columns to a thread, 32 apart, a warp to a group: element loads and stores that still coalesce
// 8192 rows of 5120 columns, all in BF16, take 64 us, 5.9 TB/s (a CTA to a row without the ring 76, three or four CTAs of
// 64 or 48 registers 64 and 65, five of 40 registers 107; three rows ahead instead of two 69).  2048 rows without a
// residual, whose 21 MB come from L2, take 13.4 us, and 6.0 more for every 1024: three CTAs need 2.6 us to a row each, for
// its chain from the copy to the codes and for their instructions, half of an SM's issue slots (2048 rows 11.3 us with
// codes from y in single FP32 numbers, whose error against FP64 was 1.1 to 1.5 times as large).

#include <algorithm>
#include <atomic>

#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace rn {

constexpr int G = 128;
constexpr int MAX_DEPTH = 2;
constexpr int RING_BYTES = 200 * 1024;

// `bytes` (a multiple of 16) from global to shared memory, both on 16-byte boundaries.
MOE_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

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

// 8 consecutive elements on a 16-byte boundary
MOE_DEV void load8(const void* p, int64_t i, bool bf16, float (&v)[8]) {
  if (bf16) {
    const uint4 a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(w[j]);
      v[2 * j + 1] = bf16_hi(w[j]);
    }
  } else {
    const float4* a = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 f = a[j];
      v[4 * j] = f.x;
      v[4 * j + 1] = f.y;
      v[4 * j + 2] = f.z;
      v[4 * j + 3] = f.w;
    }
  }
}
MOE_DEV void store8(void* p, int64_t i, bool bf16, const float (&v)[8]) {
  if (bf16) {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    float4* a = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    a[0] = make_float4(v[0], v[1], v[2], v[3]);
    a[1] = make_float4(v[4], v[5], v[6], v[7]);
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

// h of N columns to y and codes; LANES neighbouring lanes hold a group of 128.  Returns the group's scale.
template <int N, int LANES>
MOE_DEV float finish(float (&h)[N], const float (&w)[N], float inv, uint32_t (&codes)[N / 4]) {
  float lo[N], v[N];  // h w = h + lo from here on
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = h[i] * w[i];
    lo[i] = __fmaf_rn(h[i], w[i], -t);
    h[i] = t;
    m = max(m, __float_as_uint(t) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float most = __uint_as_float(m), amax = most * inv;
  float scale;
  // in pairs, where nothing overflows or is rounded to a subnormal, and y's floor of 2^-100 is not the scale's
  if (most > 0x1p-60f && most < 0x1p100f && amax > __uint_as_float(kFp8AmaxFloorBits) && amax < 0x1p100f) {
    // 448 / most = b + bl to 2^-44, a quotient of double length: the remainder of an approximate one, exact in an FMA, by
    // the reciprocal again (Dekker, A floating-point technique for extending the available precision, 1971)
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(most));  // (to 2^-23)
    const float b = 448.f * r, bl = __fmaf_rn(-b, most, 448.f) * r;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fmaf_rn(h[i], b, __fmaf_rn(h[i], bl, lo[i] * b));
    // amax / 448, the quotient by the rounded reciprocal corrected with its remainder (Markstein, Computation of elementary
    // functions on the IBM RISC System/6000 processor, 1990): the nearest number for every amax here
    const float s = amax * (1.f / 448.f);
    scale = __fmaf_rn(__fmaf_rn(-448.f, s, amax), 1.f / 448.f, s);
  } else {
    float by;
    fp8_scale(__float_as_uint(amax) & 0x7FFFFFFFu, scale, by);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = h[i] * inv * by;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) h[i] *= inv;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) codes[i] = pack_e4m3x4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  return scale;
}

MOE_DEV float inverse_root(const RmsNormArgs& a, float sum) {
  return __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)a.K) + a.eps));
}

// C pieces of twice 8 columns to a thread.  depth > 0: that many rows of shared memory.
template <int C>
__global__ void __maxnreg__(C == 1 ? 64 : 128) ring_kernel(RmsNormArgs a, int depth, int x_bytes, int r_bytes) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[MAX_DEPTH];
  __shared__ float s_part[2][32];
  __shared__ int s_abort;
  const int threads = blockDim.x, tid = threadIdx.x, lane = tid & 31, warps = threads >> 5, n_rows = gridDim.x;
  if (tid == 0) {
    for (int i = 0; i < depth; ++i) mbar_init(smem_u32(&full[i]), 1);
    s_abort = 0;
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  const uint8_t* x = static_cast<const uint8_t*>(a.x);
  const uint8_t* r = static_cast<const uint8_t*>(a.r);
  const int64_t x_pitch = a.ld_x * (a.x_bf16 ? 2 : 4), r_pitch = a.ld_r * (a.r_bf16 ? 2 : 4);
  auto fetch = [&](int64_t row, int slot) {  // one thread
    const uint32_t at = smem_u32(ring) + slot * (x_bytes + r_bytes), bar = smem_u32(&full[slot]);
    mbar_arrive_expect_tx(bar, x_bytes + r_bytes);
    bulk_load(at, x + row * x_pitch, x_bytes, bar);
    if (r_bytes > 0) bulk_load(at + x_bytes, r + row * r_pitch, r_bytes, bar);
  };
  if (tid == 0)
    for (int i = 0; i < depth; ++i)
      if ((int64_t)blockIdx.x + i * n_rows < a.R) fetch((int64_t)blockIdx.x + i * n_rows, i);
  __syncthreads();
  auto column = [&](int c, int half) {
    const int p = c * threads + tid;
    return p / 8 * G + p % 8 * 8 + half * 64;
  };
  int slot = 0, parity = 0, part = 0;
  bool live = true;  // no wait has run out
  for (int64_t row = blockIdx.x; row < a.R; row += n_rows) {
    const void *xs = x + row * x_pitch, *rs = r + row * r_pitch;
    if (depth > 0) {
      // (a row whose wait ran out has wrong values, and the error is set; no row is fetched from then on, as its slot may
      // be one that is still waited for)
      live &= mbar_wait_warp(smem_u32(&full[slot]), parity, &s_abort, a.err, a.wait_ns);
      xs = ring + slot * (x_bytes + r_bytes);
      rs = ring + slot * (x_bytes + r_bytes) + x_bytes;
    }
    float h[C][16];
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = column(c, half);
        float v[8] = {}, u[8] = {};
        if (k < a.K) {
          load8(xs, k, a.x_bf16, v);
          if (a.r != nullptr) load8(rs, k, a.r_bf16, u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = v[i] + u[i];
          h[c][half * 8 + i] = t;
          sum = __fmaf_rn(t, t, sum);
        }
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_part[part][tid >> 5] = sum;
    __syncthreads();  // (the row's sums are there, its shared memory is read, and the parts of the row before it)
    if (depth > 0) {
      if (tid == 0 && live && row + depth * n_rows < a.R) fetch(row + depth * n_rows, slot);
      if (++slot == depth) {
        slot = 0;
        parity ^= 1;
      }
    }
    sum = s_part[part][0];
    for (int i = 1; i < warps; ++i) sum += s_part[part][i];
    part ^= 1;
    const float inv = inverse_root(a, sum);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float w[16];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = column(c, half);
        float v[8] = {}, u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = h[c][half * 8 + i];
        if (k < a.K) {
          load8(a.w, k, a.w_bf16, v);
          if (a.r != nullptr) store8(a.h, row * a.ld_h + k, a.r_bf16, u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) w[half * 8 + i] = v[i];
      }
      uint32_t codes[4];
      const float scale = finish<16, 8>(h[c], w, inv, codes);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = column(c, half);
        if (k >= a.K) continue;
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = h[c][half * 8 + i];
        if (a.y != nullptr) store8(a.y, row * a.ld_y + k, true, u);
        *reinterpret_cast<uint2*>(a.q + row * a.ld_q + k) = make_uint2(codes[2 * half], codes[2 * half + 1]);
        if ((lane & 7) == 0 && half == 0) a.s[row * a.s_row + k / G * a.s_grp] = scale;
      }
    }
  }
  if (tid == 0 && !live)
    for (int i = 0; i < depth; ++i) {  // no copy may still be on its way into a CTA that is gone
      mbar_wait_drain(smem_u32(&full[i]), 0);
      mbar_wait_drain(smem_u32(&full[i]), 1);
    }
}

// A CTA to a row, or (rows of one warp) a warp to a row.  C: groups to a warp.
template <int C>
__global__ void __launch_bounds__(512) any_kernel(RmsNormArgs a, int warps) {
  __shared__ float s_part[32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_cta = warps == 1 ? (int)(blockDim.x >> 5) : 1;
  const int64_t row = (int64_t)blockIdx.x * per_cta + (warps == 1 ? warp : 0);
  if (row >= a.R) return;  // (whole warps, and only where no barrier follows)
  float h[C][4];
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k0 = (c * warps + (warps == 1 ? 0 : warp)) * G + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 32 * i;
      h[c][i] = k < a.K ? load1(a.x, row * a.ld_x + k, a.x_bf16) : 0.f;
      if (a.r != nullptr && k < a.K) h[c][i] += load1(a.r, row * a.ld_r + k, a.r_bf16);
      sum = __fmaf_rn(h[c][i], h[c][i], sum);
    }
  }
  sum = row_sum(sum, s_part, warps);
  const float inv = inverse_root(a, sum);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int grp = c * warps + (warps == 1 ? 0 : warp), k0 = grp * G + lane;
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 32 * i;
      w[i] = k < a.K ? load1(a.w, k, a.w_bf16) : 0.f;
      if (a.r != nullptr && k < a.K) store1(a.h, row * a.ld_h + k, h[c][i], a.r_bf16);
    }
    uint32_t codes[1];
    const float scale = finish<4, 32>(h[c], w, inv, codes);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 32 * i;
      if (k >= a.K) continue;
      if (a.y != nullptr) store1(a.y, row * a.ld_y + k, h[c][i], true);
      a.q[row * a.ld_q + k] = (uint8_t)(codes[0] >> (8 * i));
    }
    if (lane == 0 && grp * G < a.K) a.s[row * a.s_row + grp * a.s_grp] = scale;
  }
}

bool wide(const void* p, int64_t ld, bool bf16) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (bf16 ? 2 : 4) % 16 == 0;
}

template <int C>
int launch_ring(const RmsNormArgs& a, cudaStream_t st) {
  const int nsm = device_sm_count(), dev = current_device_index();
  if (nsm <= 0 || dev < 0) return MOE_ERR_CUDA;
  const int threads = ((a.K + G - 1) / G * 8 + 32 * C - 1) / (32 * C) * 32;
  const int x_bytes = a.K * (a.x_bf16 ? 2 : 4), r_bytes = a.r != nullptr ? a.K * (a.r_bf16 ? 2 : 4) : 0;
  // CTAs of an SM (64 registers a thread, 128 for the longest rows), and their share of its shared memory (rows past it are read without the ring)
  const int per_sm = std::max(1, std::min(16, (C == 1 ? 1024 : 512) / threads));
  const int depth = std::min(MAX_DEPTH, RING_BYTES / per_sm / (x_bytes + r_bytes));
  static std::atomic<uint64_t> configured{0};  // a bit per device
  if (!(configured.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    if (cudaFuncSetAttribute(ring_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES) != cudaSuccess)
      return MOE_ERR_CUDA;
    configured.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  }
  return launch_pdl(ring_kernel<C>, dim3(std::min(a.R, per_sm * nsm)), dim3(threads), depth * (x_bytes + r_bytes), st, a, depth,
                    x_bytes, r_bytes);
}

template <int C>
int launch_any(const RmsNormArgs& a, int warps, cudaStream_t st) {
  const int per_cta = warps == 1 ? 4 : 1;  // (rows of one warp: four to a CTA)
  return launch_pdl(any_kernel<C>, dim3((a.R + per_cta - 1) / per_cta), dim3(32 * warps * per_cta), 0, st, a, warps);
}

}  // namespace rn

int rms_norm_launch(const RmsNormArgs& a, cudaStream_t st) {
  using namespace rn;
  const bool ring = a.K % 8 == 0 && wide(a.x, a.ld_x, a.x_bf16) && wide(a.w, 0, a.w_bf16) &&
                    (a.r == nullptr || (wide(a.r, a.ld_r, a.r_bf16) && wide(a.h, a.ld_h, a.r_bf16))) &&
                    (a.y == nullptr || wide(a.y, a.ld_y, true));
  if (ring) {
    if (a.K <= 64 * G) return launch_ring<1>(a, st);
    if (a.K <= 128 * G) return launch_ring<2>(a, st);
    return launch_ring<4>(a, st);
  }
  const int groups = (a.K + G - 1) / G;
  if (groups <= 16) return launch_any<1>(a, groups, st);
  if (groups <= 64) return launch_any<4>(a, (groups + 3) / 4, st);
  return launch_any<16>(a, (groups + 15) / 16, st);
}

}  // namespace moe
