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

// silu(min(g, L)) * clamp(u, -L, L) of FP32 sums, NaN kept.  silu(z) = z / (1 + e^-z).
//
// FAST: e^-z by the hardware's approximate power of two (2^-22 relative) and the quotient by its approximate
// reciprocal (2^-23), for the wide kernel, whose epilogue nothing hides: with the accurate forms the gate/up
// product of 256 tokens at 64 experts takes 65.8 us against 41.9, of 2048 tokens at 40 experts 326 against 287.
// The power's argument t = fl(-z log2 e) is off by up to 2^-24 |t|, which alone would make 2^-18 of e^-z at
// z = -64 (41.1 and 284 us).  What it misses, x = -z - t ln 2, is exact to 2^-28 |t| in one FMA (ln 2
// rounded), and e^-z = 2^t (1 + x) to within x^2 / 2 < 2^-35: in all 2^-20 of the result, 2^-21 with the
// accurate forms.  t is kept within +-127, so that neither 2^t nor x overflows: where it is more, 2^t (1 + x)
// is past 2^126 and its reciprocal is flushed to zero (the result to a zero, the limit of silu), where it is
// less, 2^t is flushed and the reciprocal 1.
template <bool FAST>
MOE_DEV float swiglu_keep_nan(float g, float u, float L) {
  const float gm = min_nan(g, L);
  const float uc = max_nan(min_nan(u, L), -L);
  if (!FAST) return __fdiv_rn(gm, 1.0f + expf(-gm)) * uc;
  const float t = fmaxf(fminf(gm * -1.44269504f, 127.0f), -127.0f);
  const float x = __fmaf_rn(t, -0.693147181f, -gm);
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fmaf_rn(e, x, 1.0f + e)));
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
