// fp8.cuh -- device helpers shared by the FP8 (E4M3, 128-element scales) kernels.
#pragma once

#include "common.cuh"

namespace moe {

constexpr uint32_t kFp8AmaxFloorBits = 0x0D800000u;  // 2^-100

// Scale and its reciprocal of a group whose largest magnitude has the bits amax_bits (inf and NaN
// compare above every number): a = max(amax, 2^-100), scale = a / 448, inv = 448 (1 / a), the form in which
// PyTorch evaluates 448 / a, so that its codes are these; both NaN for a group with a value that is not
// finite.
MOE_DEV void fp8_scale(uint32_t amax_bits, float& scale, float& inv) {
  const bool finite = amax_bits < 0x7F800000u;
  const float a = __uint_as_float(finite ? max(amax_bits, kFp8AmaxFloorBits) : 0x7FC00000u);
  scale = __fdiv_rn(a, 448.0f);
  inv = 448.0f * __frcp_rn(a);
}

// Four floats to E4M3 codes, round to nearest even, a in the low byte.
MOE_DEV uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint32_t out;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}"
      : "=r"(out)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return out;
}

// Minimum and maximum that keep a NaN (fminf and fmaxf drop it), one instruction each.
MOE_DEV float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
MOE_DEV float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// silu(min(g, L)) * clamp(u, -L, L) of FP32 sums, NaN kept.  silu(z) = z / (1 + e^-z).  FAST: with the
// hardware's approximate power of two and reciprocal (2^-22 and 2^-23 relative, against 2^-24 of FP32: the
// result is rounded to four bits, and one in about a million values then to the other neighbour), for
// kernels in which the accurate forms' instructions count.  For z -> -inf the power overflows and the
// quotient is -0, the limit of silu.
template <bool FAST>
MOE_DEV float swiglu_keep_nan(float g, float u, float L) {
  const float gm = min_nan(g, L);
  const float uc = max_nan(min_nan(u, L), -L);
  if (!FAST) return __fdiv_rn(gm, 1.0f + expf(-gm)) * uc;
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(gm * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return gm * r * uc;
}

// Load from the shared memory of CTA `rank` of the cluster, at the offset of local_addr in ours.
MOE_DEV float ld_shared_cluster_f32(uint32_t local_addr, uint32_t rank) {
  uint32_t ra;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(local_addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra) : "memory");
  return v;
}

}  // namespace moe
