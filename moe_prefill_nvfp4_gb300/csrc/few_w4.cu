// few_tokens.cu -- a whole layer of routed experts (and a shared one) for at most 16 tokens, in two launches:
//
//   out[t] = sum_s wts[t, s] * W_dn[e] act(W_gu[e] x[t])  (+ shared),  e = ids[t, s],
//   act = silu(min(g, L)) * clamp(u, -L, L)
//
// for experts in block-scaled FP8 (rows and activations quantised to E4M3, 128 columns to a scale) or in NVFP4
// (rows and activations in FP16 times a power of two per 128 columns).
//
// Bound by the weights' bytes: of each expert that a token has picked, once.  So everything else is kept out of
// their way:
//   prep  router logits (a CTA to an expert and eight tokens), the tokens' rows quantised, counters to zero.
//   few   persistent, a CTA to an SM.  Each CTA routes the few tokens by itself (logits -> picks -> list of the
//         picked experts: the same in all CTAs), which is shorter than a launch.  Then every warp but one works for
//         itself: it draws units from a counter, first all experts' gate/up units, then all experts' down units, and
//         streams their weights through a small ring of its own, steps ahead of its products and across units.
//         Because weights depend on no result, the streams run on into the down units while the activations that those
//         need are still being made.  Experts are drawn in the same order in both halves, so an expert's activations
//         are long finished when its down units come, but for the last ones.
//
// A unit is 32 weight rows (16 gate rows with their up rows, or 32 down rows) over a slice of k.  The products are
// warp-level tensor-core ones: the weight rows are the M operand, the expert's tokens the N operand (8 columns, or
// 16), and sums over slices are added up later, in order, by whoever finishes what they belong to: the last of the
// units of 128 activations makes the activations and quantises them, the last of the units of 32 output columns
// adds up slices and experts.  No sum depends on who was last.
//
// What bounds it beside the memory is instructions: an SM has 2070 cycles for 45 KB, and a step of 4 KB takes a warp
// some 200.  Forms that shared a unit's k among the warps of a CTA spent as many again on handing over: one warp
// that loads for eight that multiply 61 us for one token at 160 experts, eight that load for themselves and hand
// their sums to a ninth 74 us.  (tcgen05 would take the codes from shared memory without conversions, but 128 weight
// rows at a time, which are 640 KB of a gate/up tile and have to be cut along k for 152 SMs all the same.)
//
// A unit's dependencies are all drawn before it, so whichever CTAs are running make progress, also beside
// another call's kernel that holds a part of the SMs.  Every wait is bounded (MOE_DEVERR_TIMEOUT).

#include <algorithm>
#include <atomic>

#include <cuda_fp16.h>

#include "few.h"
#include "fp8.cuh"
#include "internal.h"
#include "topk.cuh"

namespace moe {
namespace few_w4 {

constexpr int G = 128;             // columns of a scale
constexpr int GROUP_BYTES = 256;   // of an activation row
constexpr int ROWS = 32;           // weight rows of a unit, two MMA tiles
constexpr int HALF = ROWS / 2;     // gate rows, up rows
constexpr int PUSHED = 2;          // finished units of a worker that are not published yet
constexpr int WORKERS = 13;
constexpr int FINISHERS = 2;
constexpr int WARPS = WORKERS + 1 + FINISHERS;  // four to a quarter of the SM: 128 registers; one publishes
constexpr int THREADS = 32 * WARPS;
constexpr int MAX_T = MOE_FEW_MAX_TOKENS;
constexpr int MAX_SLOTS = MAX_T * 32;

// Activation rows are FP16 in both formats: an E4M3 code's value, or a power of two times the number.  The weights'
// codes are turned to FP16 in registers as well (one conversion to two), because a warp-level FP8 product is the same
// conversions of both operands, again for every product, and an FP16 one.
//
// A step is two groups of a unit's rows in pieces of 16 bytes: FP8 [group][32 rows][8 pieces], 8 KB, NVFP4 [32 rows][8
// pieces] of both groups, 4 KB, and their block scales, 16 bytes to a row.  Odd rows' halves of 64 bytes are swapped, so
// that the pieces that four lanes take of two neighbouring rows lie in the 32 banks once.
template <bool W4>
struct Fmt {
  static constexpr int WEIGHTS = W4 ? 4096 : 8192;
  static constexpr int STEP_BYTES = WEIGHTS + (W4 ? 512 : 0);
  static constexpr int STEPS = W4 ? 3 : 2;  // of a worker's ring
};

struct Entry {
  int expert;  // of the held ones; -1: the shared expert
  short m, first;
};

struct Smem {
  int2 pushed_unit[WORKERS][PUSHED];   // finished units: entry, place * 2 + (down)
  volatile int pushed[WORKERS], published[WORKERS];
  volatile int working;                    // workers that are not done
  int first_unit, routed, abort;
  volatile int ready;                      // the first entries whose activations are there
  float wts[MAX_SLOTS];
  short pos[MAX_SLOTS];                    // row of slot (t, s), -1: of an expert held elsewhere
  uint8_t token[MAX_SLOTS + MAX_T];        // of row p
  Entry entry[MAX_SLOTS + 2];
};
// (only before the rings are used, in their place)
struct Routing {
  int32_t ids[MAX_SLOTS];
  uint32_t tokens[MOE_FEW_MAX_EXPERTS];  // bit t: token t has picked the expert
  short first[MOE_FEW_MAX_EXPERTS];      // its first row
  int sums[WARPS];                       // of 32 experts each: rows, entries << 16
};
static_assert(MOE_FEW_MAX_EXPERTS <= 32 * WARPS && MAX_T <= WARPS, "a warp to 32 experts, and to a token");

MOE_DEV uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
MOE_DEV uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
// 16 bytes past L1
MOE_DEV void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits for the oldest of n groups of this thread's copies
MOE_DEV void copies_wait_oldest(int n) {
  if (n <= 1)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// D += A B, A 16 x 16 FP16, B 16 x 8.  Lane (g = lane / 4, t = lane % 4): a0, a2 of row g, a1, a3 of row g + 8; b of
// column g; d0, d1 row g, columns 2t, 2t + 1; d2, d3 row g + 8.  Which k a register holds is free as long as A and B
// agree.
MOE_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
MOE_DEV uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

MOE_DEV uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

MOE_DEV uint2 half4(const float (&v)[4]) {
  const __half2 lo = __floats2half2_rn(v[0], v[1]), hi = __floats2half2_rn(v[2], v[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
MOE_DEV uint2 half4(uint32_t codes) {
  uint2 v;
  e4m3x4_to_f16x2(codes, v.x, v.y);
  return v;
}

// A group of an activation row, 4 consecutive columns to a lane, in the order that the products take it.  Lane t of
// four has 16-byte pieces (8 columns): in FP8 the columns 16 t .. 16 t + 15 of each half group, as the weights' 16-byte
// pieces have them, in NVFP4 the columns 32 t .. 32 t + 31; the four lanes' i-th pieces are neighbours.
template <bool W4>
MOE_DEV void store_columns(uint2 v, uint8_t* values) {
  const int lane = threadIdx.x & 31, piece = lane >> 1;
  const int place = W4 ? (piece & 3) * 4 + (piece >> 2) : ((piece >> 3) * 2 + (piece & 1)) * 4 + (piece >> 1 & 3);
  *reinterpret_cast<uint2*>(values + place * 16 + (lane & 1) * 8) = v;
}

// A group of a row, 4 consecutive columns to a lane: its values; returns its scale.
template <bool W4>
MOE_DEV float write_group(const float (&v)[4], uint8_t* values) {
  float scale, by;
  if constexpr (W4) {
    // a power of two that brings the group's largest finite magnitude to [2^14, 2^15): FP16 then holds BF16
    // numbers down to 2^-31 of it exactly, and FP32 ones to 2^-12 of their value; what is not finite stays so
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, abs_bits(v[i]) < 0x7F800000u ? abs_bits(v[i]) : 0u);
    m = __reduce_max_sync(0xffffffffu, m);
    const int ex = max((int)(m >> 23), 27);  // biased; at least 2^-100
    scale = __uint_as_float((uint32_t)(ex - 14) << 23);
    by = __uint_as_float((uint32_t)(254 - (ex - 14)) << 23);
  } else {
    const uint32_t m = __reduce_max_sync(
        0xffffffffu, max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3]))));
    fp8_scale(m, scale, by);
  }
  float q[4] = {v[0] * by, v[1] * by, v[2] * by, v[3] * by};
  store_columns<W4>(W4 ? half4(q) : half4(pack_e4m3x4(q[0], q[1], q[2], q[3])), values);
  return scale;
}

// ------------------------------------------------------------------------------------------------
// prep: block 0 clears the counters, blocks 1 .. T quantise the tokens' rows (or take the given ones), the others
// make the router's logits, of one expert and eight tokens each

constexpr int PREP_THREADS = 256, PREP_TOKENS = 8;

template <bool W4, int TT>
__global__ void __launch_bounds__(PREP_THREADS) prep_kernel(FewArgs a) {
  __shared__ float s_part[PREP_THREADS / 32][TT];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < a.n_counters; i += PREP_THREADS) a.counters[i] = 0;
    return;
  }
  if ((int)blockIdx.x <= a.T) {
    const int t = blockIdx.x - 1, groups = a.H / G;
    if (a.rows_q != nullptr) {
      for (int g = warp; g < groups; g += PREP_THREADS / 32) {
        const uint32_t codes = reinterpret_cast<const uint32_t*>(a.rows_q + t * a.rows_ld + g * G)[lane];
        store_columns<W4>(half4(codes), a.x_made + ((size_t)t * groups + g) * GROUP_BYTES);
        if (lane == 0) a.x_scales_made[t * groups + g] = a.rows_s[t * a.rows_s_row + g * a.rows_s_grp];
      }
      return;
    }
    for (int g = warp; g < groups; g += PREP_THREADS / 32) {
      const uint2 w = *reinterpret_cast<const uint2*>(a.x + (size_t)t * a.H + g * G + lane * 4);
      const float v[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
      const float scale = write_group<W4>(v, a.x_made + ((size_t)t * groups + g) * GROUP_BYTES);
      if (lane == 0) a.x_scales_made[t * groups + g] = scale;
    }
    return;
  }
  // one expert's logits of TT tokens: its router row is read once, the tokens' rows come from the caches
  const int at = blockIdx.x - 1 - a.T, e = at % a.E, t0 = at / a.E * PREP_TOKENS;
  float acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.f;
  const uint4* w = reinterpret_cast<const uint4*>(a.w_router + (size_t)e * a.H);
  const uint4* x = reinterpret_cast<const uint4*>(a.x + (size_t)t0 * a.H);
  const int n = a.H / 8;
#pragma unroll 3
  for (int i = threadIdx.x; i < n; i += PREP_THREADS) {
    const uint4 wv = w[i];
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint4 xv = t0 + t < a.T ? x[(size_t)t * n + i] : make_uint4(0, 0, 0, 0);
      const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[t] = __fmaf_rn(bf16_lo(ww[j]), bf16_lo(xx[j]), acc[t]);
        acc[t] = __fmaf_rn(bf16_hi(ww[j]), bf16_hi(xx[j]), acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
    if (lane == 0) s_part[warp][t] = acc[t];
  }
  __syncthreads();
  if (threadIdx.x < TT && t0 + (int)threadIdx.x < a.T) {
    float v = s_part[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < PREP_THREADS / 32; ++i) v += s_part[i][threadIdx.x];
    a.logits_ws[(size_t)(t0 + threadIdx.x) * a.E + e] = v;
  }
}

// ------------------------------------------------------------------------------------------------
// few: routing

MOE_DEV int shared_entries(const FewArgs& a) { return a.Is > 0 ? (a.T + 7) / 8 : 0; }

MOE_DEV void route_rows(const FewArgs& a, Smem& s, Routing& r) {
  const float* logits = a.logits != nullptr ? a.logits : a.logits_ws;
  static_assert(MAX_T <= WARPS, "a warp to a token");
  const int t = threadIdx.x >> 5;
  if (t < a.T) {
    const float* row = logits + (size_t)t * a.E;
    int32_t* ids = r.ids + t * a.k;
    float* wts = s.wts + t * a.k;
    if (a.E <= 64)
      topk_row<2>(row, a.bias, a.E, a.k, a.renormalize, a.routed_scale, ids, wts, a.err);
    else if (a.E <= 160)
      topk_row<5>(row, a.bias, a.E, a.k, a.renormalize, a.routed_scale, ids, wts, a.err);
    else if (a.E <= 256)
      topk_row<8>(row, a.bias, a.E, a.k, a.renormalize, a.routed_scale, ids, wts, a.err);
    else
      topk_row<16>(row, a.bias, a.E, a.k, a.renormalize, a.routed_scale, ids, wts, a.err);
  }
}

// The list of the picked experts that are held here, in expert order, and their rows, in token order: row p of
// an entry is row p of the activations and of Y.  An expert of more than 8 tokens is two entries (8 are the columns of
// an MMA; the second entry finds the weights in L2).  A shared expert is the first one or two, with rows T k ..
// T k + T - 1.  r.tokens is zero before.
template <bool W4>
MOE_DEV void make_entries(const FewArgs& a, Smem& s, Routing& r) {
  const int slots = a.T * a.k, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  route_rows(a, s, r);
  __syncthreads();
  for (int i = tid; i < slots; i += THREADS) {
    const int e = r.ids[i];
    const bool held = W4 ? a.w4[0].packed[e] != nullptr && a.w4[1].packed[e] != nullptr
                         : e >= a.first && e < a.first + a.count;
    if (held) atomicOr(&r.tokens[e], 1u << (i / a.k));
  }
  __syncthreads();
  const int sh = shared_entries(a), e = tid;
  const uint32_t mine = e < a.E ? r.tokens[e] : 0u;
  const int m = __popc(mine);
  int sums = m | (m + 7) / 8 << 16;  // rows and entries, inclusive prefixes over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += v;
  }
  if (lane == 31) r.sums[warp] = sums;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += r.sums[w];
    all += r.sums[w];
  }
  if (m > 0) {
    before += sums - (m | (m + 7) / 8 << 16);
    const int first = before & 0xFFFF, n = sh + (before >> 16);
    r.first[e] = (short)first;
    s.entry[n] = Entry{e - a.first, (short)min(m, 8), (short)first};
    if (m > 8) s.entry[n + 1] = Entry{e - a.first, (short)(m - 8), (short)(first + 8)};
    int q = first;
    for (uint32_t b = mine; b != 0; b &= b - 1) s.token[q++] = (uint8_t)(__ffs(b) - 1);
  }
  if (tid == 0) {
    s.routed = all >> 16;
    for (int i = 0; i < sh; ++i) s.entry[i] = Entry{-1, (short)min(8, a.T - 8 * i), (short)(slots + 8 * i)};
  }
  if (sh > 0 && tid < a.T) s.token[slots + tid] = (uint8_t)tid;
  __syncthreads();
  for (int i = tid; i < slots; i += THREADS) {
    const uint32_t of = r.tokens[r.ids[i]];
    s.pos[i] = of != 0 ? (short)(r.first[r.ids[i]] + __popc(of & ((1u << (i / a.k)) - 1))) : (short)-1;
  }
  __syncthreads();
}

// The next number, in lane 0.  (In one piece of assembly: the compiler would add up a warp's atomics, or choose
// between the answer and a constant for the other lanes, and wait for the answer to do so, some 2000 cycles.)
MOE_DEV int draw(int* p) {
  int v;
  asm volatile(
      "{\n .reg .pred p;\n .reg .u32 l;\n mov.u32 l, %%laneid;\n setp.eq.u32 p, l, 0;\n"
      " @p atom.relaxed.gpu.global.add.s32 %0, [%1], 1;\n}"
      : "=r"(v)
      : "l"(p)
      : "memory");
  return v;
}

// ------------------------------------------------------------------------------------------------
// few: units

// The units, in the order in which they are drawn: of each entry (the shared expert, then the routed ones) its gate/up
// units, by rows, then by slices of k, and some entries behind its down units: `lag` entries after the entry that has
// all its gate/up units drawn its activations are there, and at the end the down units of as many are left to work on
// while the last entry's activations are made.
struct Units {
  int sh, shared, total, per_shared, per_gu, per_down, lag, ahead, both, behind;
  MOE_DEV Units(const FewArgs& a, int routed) {
    sh = shared_entries(a);
    per_gu = a.I / HALF * a.slices[0];
    per_down = a.H / ROWS * a.slices[1];
    per_shared = a.Is / HALF * a.slices[0];
    shared = sh * per_shared;
    lag = min(a.lag, routed);
    ahead = shared + lag * per_gu + sh * per_down;  // all before the first routed entry's down units
    both = per_gu + per_down;
    behind = ahead + (routed - lag) * both;         // then down units only
    total = behind + lag * per_down;
  }
};

// A unit for the warp that works on it.
struct Unit {
  int entry, m, first;  // its list entry, with its rows
  int place;            // of its rows among the entry's
  int slice, grp, end;  // its groups
  bool down, shared;
};

MOE_DEV Unit unit_at(const FewArgs& a, const Smem& s, const Units& us, int u) {
  Unit un;
  int v = u;
  un.entry = 0;
  un.down = false;
  if (u >= us.ahead) {
    const bool last = u >= us.behind;
    const int per = last ? us.per_down : us.both;
    v -= last ? us.behind : us.ahead;
    const int i = v / per;
    v -= i * per;
    un.down = last || v < us.per_down;
    un.entry = us.sh + i + (last ? s.routed - us.lag : un.down ? 0 : us.lag);
    if (!un.down) v -= us.per_down;
  } else if (u >= us.shared) {
    v -= us.shared;
    un.down = v >= us.lag * us.per_gu;  // the shared expert's
    if (un.down) {
      v -= us.lag * us.per_gu;
      un.entry = v >= us.per_down;
      v -= un.entry * us.per_down;
    } else {
      const int i = v / us.per_gu;
      v -= i * us.per_gu;
      un.entry = us.sh + i;
    }
  } else {
    un.entry = v >= us.per_shared;
    v -= un.entry * us.per_shared;
  }
  const Entry en = s.entry[un.entry];
  un.m = en.m;
  un.first = en.first;
  un.shared = en.expert < 0;
  const int slices = un.down ? a.slices[1] : a.slices[0], each = un.down ? a.slice_groups[1] : a.slice_groups[0];
  un.place = v / slices;
  un.slice = v - un.place * slices;
  const int groups = (un.down ? (un.shared ? a.Is : a.I) : a.H) / G;
  un.grp = un.slice * each;
  un.end = min(groups, un.grp + each);  // (<= grp: another expert has more slices; its sums are zeros)
  return un;
}

// A group of activation rows as the MMAs take them, for 8 tokens, with its scales.
struct Columns {
  uint4 b[4];
  float sa[2];
  float sw[2];  // FP8: the weight's, of the unit's first and second rows
};

// One group of 16 weight rows: sum of the codes' products.
MOE_DEV void tile_fp8(uint32_t rows_at, const Columns& x, float (&sum)[4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t piece = rows_at + g * 128 + (((q * 4 + t) ^ ((g & 1) << 2)) << 4);
    const uint4 lo = lds128(piece), hi = lds128(piece + 1024);
    const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 al = half4(l[i]), au = half4(u[i]);
      const uint4 b = x.b[2 * q + (i >> 1)];
      mma_f16(sum, al.x, au.x, al.y, au.y, i & 1 ? b.z : b.x, i & 1 ? b.w : b.y);
    }
  }
}
// 32 consecutive k to a lane (16 bytes of each row), 8 to a word: two MMAs
MOE_DEV void tile_w4(uint32_t rows_at, uint32_t scales_at, int j, const Columns& x, float (&sum)[4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
  const uint32_t piece = rows_at + g * 128 + (((j * 4 + t) ^ ((g & 1) << 2)) << 4);
  const uint4 lo = lds128(piece), hi = lds128(piece + 1024);
  const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u[4] = {hi.x, hi.y, hi.z, hi.w};
  const uint32_t scale = scales_at + g * 16 + j * 8 + t * 2;
  uint32_t sl, su, unused;
  e4m3x4_to_f16x2(lds_u16(scale), sl, unused);
  e4m3x4_to_f16x2(lds_u16(scale + 128), su, unused);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t al[4], au[4];
    e2m1x8_to_f16x2(l[q], al);
    e2m1x8_to_f16x2(u[q], au);
    const uint32_t both_l = prmt(sl, sl, q < 2 ? 0x1010 : 0x3232), both_u = prmt(su, su, q < 2 ? 0x1010 : 0x3232);
#pragma unroll
    for (int v = 0; v < 4; ++v) {  // exact: at most 6 bits
      al[v] = mul_f16x2(al[v], both_l);
      au[v] = mul_f16x2(au[v], both_u);
    }
    mma_f16(sum, al[0], au[0], al[1], au[1], x.b[q].x, x.b[q].y);
    mma_f16(sum, al[2], au[2], al[3], au[3], x.b[q].z, x.b[q].w);
  }
}

// Waits for a count of what other warps have stored and published.
MOE_DEV bool wait_count(const FewArgs& a, Smem& s, const int* count, int need) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    uint64_t t0 = 0;
    for (int n = 1;; ++n) {
      int v;
      asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
      if (v >= need) break;
      ok = !*(volatile int*)&s.abort;
      if (!ok) break;
      if (n % 64 == 0) {  // (a poll is a round trip to L2)
        if (t0 == 0) t0 = globaltimer_ns();
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          s.abort = 1;
          set_error(a.err, MOE_DEVERR_TIMEOUT);
        }
      }
      __nanosleep(50);
    }
  }
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok;
}

// Waits until the entry's activations are there, as the publisher has seen it.
MOE_DEV bool wait_ready(const FewArgs& a, Smem& s, int entry) {
  const volatile int& ready = s.ready;
  bool ok = true;
  if (ready <= entry) {
    uint64_t t0 = 0;
    for (int n = 1; ready <= entry; ++n) {
      if (*(volatile int*)&s.abort) {
        ok = false;
        break;
      }
      if (n % 1024 == 0) {
        if (t0 == 0) t0 = globaltimer_ns();
        if (globaltimer_ns() - t0 > 2 * kWaitLimitNs) {
          s.abort = 1;
          set_error(a.err, MOE_DEVERR_TIMEOUT);
        }
      }
      __nanosleep(20);
    }
  }
  __threadfence_block();
  return __all_sync(0xffffffffu, ok);
}

// All units of 128 activations of an entry are stored: the whole warp adds up their slices, and makes the activations
// and quantises them for the down products.
template <bool W4>
MOE_DEV void finish_group(const FewArgs& a, Smem& s, int entry, int grp) {
  const int lane = threadIdx.x & 31;
  const Entry en = s.entry[entry];
  const bool is_shared = en.expert < 0;
  const int inter = is_shared ? a.Is : a.I, groups = inter / G, first = en.first - (is_shared ? a.T * a.k : 0);
  const float limit = is_shared ? a.shared_limit : a.limit;
  const size_t slice = (size_t)(is_shared ? a.T : a.T * a.k) * 2 * inter;
  const float* gu = (is_shared ? a.gu_shared : a.gu) + (size_t)first * 2 * inter + grp * G + lane * 4;
  uint8_t* values = (is_shared ? a.act_codes_shared : a.act_codes) + ((size_t)first * groups + grp) * GROUP_BYTES;
  float* scales = (is_shared ? a.act_scales_shared : a.act_scales) + (size_t)first * groups + grp;
  for (int r = 0; r < en.m; ++r) {
    float4 gate = make_float4(0.f, 0.f, 0.f, 0.f), up = gate;
    for (int i0 = 0; i0 < a.slices[0]; i0 += 4) {
      float4 p[4], q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < a.slices[0]) {
          const float* at = gu + (i0 + i) * slice + (size_t)r * 2 * inter;
          p[i] = __ldcg(reinterpret_cast<const float4*>(at));
          q[i] = __ldcg(reinterpret_cast<const float4*>(at + inter));
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < a.slices[0]) {
          gate = make_float4(gate.x + p[i].x, gate.y + p[i].y, gate.z + p[i].z, gate.w + p[i].w);
          up = make_float4(up.x + q[i].x, up.y + q[i].y, up.z + q[i].z, up.w + q[i].w);
        }
    }
    const float v[4] = {swiglu_keep_nan<false>(gate.x, up.x, limit), swiglu_keep_nan<false>(gate.y, up.y, limit),
                        swiglu_keep_nan<false>(gate.z, up.z, limit), swiglu_keep_nan<false>(gate.w, up.w, limit)};
    const float scale = write_group<W4>(v, values + (size_t)r * groups * GROUP_BYTES);
    if (lane == 0) scales[(size_t)r * groups] = scale;
  }
  __syncwarp();
  if (lane == 0) {
    __threadfence();
    counter_add_release(a.ready + entry, 1);
  }
}

// All units of 32 columns of the result are stored: the whole warp adds up slices and experts, a lane to a column,
// of several tokens at once (their loads take a round trip to L2).
template <int TOKENS, int SLOTS>
MOE_DEV void finish_columns(const FewArgs& a, Smem& s, int place) {
  const int h = place * ROWS + (threadIdx.x & 31);
  for (int t0 = 0; t0 < a.T; t0 += TOKENS) {
    float v[TOKENS];
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) v[t] = 0.f;
    for (int c0 = 0; c0 < a.k; c0 += SLOTS) {
      float sum[TOKENS][SLOTS];
      const float* at[TOKENS][SLOTS];
#pragma unroll
      for (int t = 0; t < TOKENS; ++t)
#pragma unroll
        for (int c = 0; c < SLOTS; ++c) {
          const int p = t0 + t < a.T && c0 + c < a.k ? s.pos[(t0 + t) * a.k + c0 + c] : -1;
          at[t][c] = p >= 0 ? a.Y + (size_t)p * a.H + h : nullptr;
          sum[t][c] = 0.f;
        }
#pragma unroll 2
      for (int i = 0; i < a.slices[1]; ++i) {
        float y[TOKENS][SLOTS];
#pragma unroll
        for (int t = 0; t < TOKENS; ++t)
#pragma unroll
          for (int c = 0; c < SLOTS; ++c) y[t][c] = at[t][c] != nullptr ? __ldcg(at[t][c] + i * a.y_slice) : 0.f;
#pragma unroll
        for (int t = 0; t < TOKENS; ++t)
#pragma unroll
          for (int c = 0; c < SLOTS; ++c) sum[t][c] += y[t][c];
      }
#pragma unroll
      for (int t = 0; t < TOKENS; ++t)
#pragma unroll
        for (int c = 0; c < SLOTS; ++c)
          if (at[t][c] != nullptr) v[t] = __fmaf_rn(s.wts[(t0 + t) * a.k + c0 + c], sum[t][c], v[t]);
    }
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
      if (t0 + t >= a.T) break;
      if (a.Is > 0)
        for (int i = 0; i < a.slices[1]; ++i) v[t] += __ldcg(a.Y + (size_t)(a.T * a.k + t0 + t) * a.H + h + i * a.y_slice);
      const size_t o = (size_t)(t0 + t) * a.H + h;
      if (a.shared_out != nullptr) v[t] += __bfloat162float(__ushort_as_bfloat16(a.shared_out[o]));
      a.out[o] = __bfloat16_as_ushort(__float2bfloat16_rn(v[t]));
    }
  }
}

// One worker: its units, one after another.
template <bool W4>
MOE_DEV void work(const FewArgs& a, Smem& s, uint32_t ring) {
  using F = Fmt<W4>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, me = threadIdx.x >> 5;
  ring += me * (F::STEPS * F::STEP_BYTES);
  const Units us(a, s.routed);
  // this lane's pieces of a step: one of every fourth row
  const int my_row = lane >> 3, my_piece = lane & 7;
  const uint32_t my_place = my_row * 128 + ((my_piece ^ ((my_row & 1) << 2)) << 4);
  // what is loaded next: the rest of a unit, its rows' addresses
  int next = s.first_unit + me, drawn = draw(a.counters);
  int i_grp = 0, i_end = 0, i_place = 0, loaded = 0;
  const uint8_t *first = nullptr, *second = nullptr;
  [[maybe_unused]] const uint8_t* block_scales = nullptr;
  int64_t every = 0;
  int queue[2] = {-1, -1};  // units that are being loaded or multiplied: the products', the loads'
  auto stream = [&]() {
    while (loaded < F::STEPS) {
      if (i_grp >= i_end) {
        if (queue[1] >= 0 || next >= us.total) return;  // (the products are a unit behind at most)
        const int u = next;
        next = __shfl_sync(0xffffffffu, drawn, 0);
        drawn = draw(a.counters);
        queue[1] = u;
        const Unit in = unit_at(a, s, us, u);
        i_grp = in.grp;
        i_end = in.end;
        const int inter = in.shared ? a.Is : a.I, e = max(s.entry[in.entry].expert, 0);
        const int row = in.place * (in.down ? ROWS : HALF), apart = in.down ? HALF : inter;
        int64_t ld;
        if constexpr (W4) {
          ld = (in.down ? inter : a.H) / 2;
          first = static_cast<const uint8_t*>((in.down ? a.w4[1].packed : a.w4[0].packed)[a.first + e]) + i_grp * 64;
          block_scales = static_cast<const uint8_t*>((in.down ? a.w4[1].scales : a.w4[0].scales)[a.first + e]) +
                         (row + (lane >> 4) * apart + (lane & 15)) * (ld / 8) + i_grp * 8;
        } else {
          const FewFp8Weight& w = in.shared ? (in.down ? a.w8s[1] : a.w8s[0]) : in.down ? a.w8[1] : a.w8[0];
          ld = w.ld;
          first = w.q + e * w.expert_stride + i_grp * 128;
        }
        first += (row + my_row) * ld + my_piece * 16;
        second = first + apart * ld;
        every = 4 * ld;
        continue;
      }
      const uint32_t to = ring + i_place * F::STEP_BYTES + my_place;
      const uint8_t *p = first, *q = second;
#pragma unroll
      for (int i = 0; i < HALF / 4; ++i) {
        copy16_async(to + i * 512, p);
        copy16_async(to + 2048 + i * 512, q);
        if (!W4 && i_grp + 1 < i_end) {
          copy16_async(to + 4096 + i * 512, p + 128);
          copy16_async(to + 6144 + i * 512, q + 128);
        }
        p += every;
        q += every;
      }
      if constexpr (W4) {
        copy16_async(ring + i_place * F::STEP_BYTES + F::WEIGHTS + lane * 16, block_scales);
        block_scales += 16;
      }
      copies_commit();
      first += W4 ? 128 : 256;
      second += W4 ? 128 : 256;
      i_grp += 2;
      ++loaded;
      if (++i_place == F::STEPS) i_place = 0;
    }
  };
  int place = 0, done = 0;

  // a unit's products
  auto products = [&](const Unit& un) {
    const int inter = un.shared ? a.Is : a.I, groups = (un.down ? inter : a.H) / G;
    // this lane's columns' rows (past the expert's last token: that one's again, whose sums are not stored)
    auto row = [&](int col) {
      const int p = un.first + min(col, un.m - 1);
      return !un.down ? (int)s.token[p] : un.shared ? p - a.T * a.k : p;
    };
    // (as distances from the first group's: registers are short)
    const uint8_t* values = (!un.down ? a.x_made : un.shared ? a.act_codes_shared : a.act_codes) + un.grp * GROUP_BYTES + t * 16;
    const float* scales = (!un.down ? a.x_scales_made : un.shared ? a.act_scales_shared : a.act_scales) + un.grp;
    const int b_at = row(g) * groups * GROUP_BYTES, sa_at[2] = {row(2 * t) * groups, row(2 * t + 1) * groups};
    [[maybe_unused]] const float* sw_at = nullptr;
    [[maybe_unused]] int sw_second = 0;
    if constexpr (!W4) {
      const int r = un.place * (un.down ? ROWS : HALF), blocks = (un.down ? a.H : 2 * inter) / G;
      sw_at = (un.shared ? (un.down ? a.w8s[1].s : a.w8s[0].s) : un.down ? a.w8[1].s : a.w8[0].s) +
              ((size_t)max(s.entry[un.entry].expert, 0) * blocks + r / G) * groups + un.grp;
      sw_second = un.down ? 0 : inter / G * groups;
    }
    float acc[2][4] = {};
    // the activations and scales of the group `ahead` of the current one
    auto fetch = [&](Columns& x, int ahead) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        x.b[q] = __ldcg(reinterpret_cast<const uint4*>(values + b_at + ahead * GROUP_BYTES + q * 64));
      x.sa[0] = __ldcg(scales + sa_at[0] + ahead);
      x.sa[1] = __ldcg(scales + sa_at[1] + ahead);
      if constexpr (!W4) {
        x.sw[0] = __ldg(sw_at + ahead);
        x.sw[1] = __ldg(sw_at + sw_second + ahead);
      }
    };
    auto multiply = [&](uint32_t at, int j, const Columns& x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum[4];
        if constexpr (W4)
          tile_w4(at + i * 2048, at + F::WEIGHTS + i * 256, j, x, sum);
        else
          tile_fp8(at + j * 4096 + i * 2048, x, sum);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][v] = __fmaf_rn(sum[v], W4 ? x.sa[v & 1] : x.sa[v & 1] * x.sw[i], acc[i][v]);
      }
    };
    // (fetched a group ahead: a round trip to L2 is longer than a group)
    Columns x, y;
    if (un.grp < un.end) fetch(x, 0);
    for (int grp = un.grp; grp < un.end; grp += 2) {
      const bool two = grp + 1 < un.end;
      if (two) fetch(y, 1);
      copies_wait_oldest(loaded);
      __syncwarp();
      const uint32_t at = ring + place * F::STEP_BYTES;
      multiply(at, 0, x);
      if (grp + 2 < un.end) fetch(x, 2);
      if (two) multiply(at, 1, y);
      values += 2 * GROUP_BYTES;
      scales += 2;
      sw_at += 2;
      if (++place == F::STEPS) place = 0;
      __syncwarp();
      --loaded;
      stream();
    }
    if constexpr (W4) {
      const float s2 = (un.down ? a.w4[1].scale2 : a.w4[0].scale2)[a.first + s.entry[un.entry].expert];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][v] *= s2;
    }
    // the slice's sums: [slice][row][2 I] or [slice][row][H]
    const int wide = un.down ? a.H : 2 * inter, at_row = un.place * (un.down ? ROWS : HALF), apart = un.down ? HALF : inter;
    float* to = (un.down ? a.Y + (size_t)un.slice * a.y_slice : un.shared ? a.gu_shared + (size_t)un.slice * a.T * wide
                                                                         : a.gu + (size_t)un.slice * a.T * a.k * wide) +
                (size_t)(un.shared && !un.down ? un.first - a.T * a.k : un.first) * wide + at_row + g;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int col = 2 * t + v;
      if (col < un.m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          to[(size_t)col * wide + i * apart] = acc[i][v];
          to[(size_t)col * wide + i * apart + 8] = acc[i][2 + v];
        }
    }
  };

  for (;;) {
    stream();
    queue[0] = queue[1];
    queue[1] = -1;
    if (queue[0] < 0) break;
    stream();
    const Unit un = unit_at(a, s, us, queue[0]);
    if (un.down && !wait_ready(a, s, un.entry)) break;
    products(un);
    __syncwarp();
    int room = 1;
    if (lane == 0) {
      if (done - s.published[me] >= PUSHED) {
        const uint64_t t0 = globaltimer_ns();
        while (room && done - s.published[me] >= PUSHED)
          if (*(volatile int*)&s.abort || globaltimer_ns() - t0 > kWaitLimitNs) room = 0;
      }
      s.pushed_unit[me][done % PUSHED] = make_int2(un.entry, un.place * 2 + (un.down ? 1 : 0));
      __threadfence_block();
      s.pushed[me] = done + 1;
    }
    ++done;
    if (!__shfl_sync(0xffffffffu, room, 0)) {
      if (lane == 0) {
        s.abort = 1;
        set_error(a.err, MOE_DEVERR_TIMEOUT);
      }
      break;
    }
  }
  copies_wait_oldest(0);  // (after a wait that ran out: no copy is on its way into a CTA that is gone)
  __syncwarp();
  if (lane == 0) {
    __threadfence_block();
    atomicSub((int*)&s.working, 1);
  }
}

// Finishes what all its units are stored of: each entry's groups of activations, then the columns of the result, drawn
// in this order.
template <bool W4>
MOE_DEV void finish(const FewArgs& a, Smem& s) {
  const int sh = shared_entries(a), entries = s.routed + sh, per_entry = a.I / G, per_shared = a.Is / G;
  const int groups_shared = sh * per_shared, groups = groups_shared + s.routed * per_entry, total = groups + a.H / ROWS;
  for (int drawn = draw(a.counters + 32);;) {
    const int u = __shfl_sync(0xffffffffu, drawn, 0);
    if (u >= total) return;
    drawn = draw(a.counters + 32);
    if (u >= groups) {
      if (!wait_count(a, s, a.columns_done + (u - groups), entries * a.slices[1])) return;
      if (a.T == 1)
        finish_columns<1, 8>(a, s, u - groups);
      else
        finish_columns<4, 4>(a, s, u - groups);
    } else {
      int v = u - groups_shared, e = 0;
      if (v < 0) {
        e = u >= per_shared;
        v = u - e * per_shared;
      } else {
        e = v / per_entry;
        v -= e * per_entry;
        e += sh;
      }
      if (!wait_count(a, s, a.group_done + e * a.groups_max + v, G / HALF * a.slices[0])) return;
      finish_group<W4>(a, s, e, v);
    }
  }
}

// Tells the other CTAs of the units that the workers have stored, a lane to a worker.  (The fence costs a round trip to
// L2, which the workers need not wait for.)  Looks for them which entries' activations are there.  Ends when the workers
// have (whose own waits are bounded).
MOE_DEV void publish(const FewArgs& a, Smem& s) {
  const int lane = threadIdx.x & 31, entries = s.routed + shared_entries(a);
  int seen = 0, ready = 0;
  for (;;) {
    // entries whose activations are there, from the first on that were not
    if (ready < entries) {
      int v = 0;
      const int e = ready + lane;
      if (e < entries) asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(a.ready + e) : "memory");
      const uint32_t there = __ballot_sync(0xffffffffu, e < entries && v >= (e < shared_entries(a) ? a.Is : a.I) / G);
      const int more = __ffs(~there) - 1;  // (-1: all 32)
      if (more != 0) {
        ready += more < 0 ? 32 : more;
        __syncwarp();
        if (lane == 0) {
          __threadfence_block();
          s.ready = ready;
        }
      }
    }
    const bool over = s.working == 0;
    __threadfence_block();
    const bool some = lane < WORKERS && s.pushed[lane] != seen;
    if (!__any_sync(0xffffffffu, some)) {
      if (__all_sync(0xffffffffu, over)) return;
      __nanosleep(40);
      continue;
    }
    if (some) {
      __threadfence_block();
      const int2 unit = s.pushed_unit[lane][seen % PUSHED];
      __threadfence();
      s.published[lane] = ++seen;
      counter_add_release(unit.y & 1 ? a.columns_done + (unit.y >> 1) : a.group_done + unit.x * a.groups_max + (unit.y >> 1) * HALF / G, 1);
    }
  }
}

template <bool W4>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ FewArgs a) {
  using F = Fmt<W4>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Smem s;
  Routing& r = *reinterpret_cast<Routing*>(smem);
  for (int e = threadIdx.x; e < a.E; e += THREADS) r.tokens[e] = 0;
  if (threadIdx.x < WORKERS) s.pushed[threadIdx.x] = s.published[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    s.working = WORKERS;
    s.ready = 0;
    s.abort = 0;
  }
  griddep_wait();
  griddep_launch_dependents();
  // (the first units of all workers at once)
  if (threadIdx.x == 0) s.first_unit = atomicAdd(a.counters, WORKERS);
  make_entries<W4>(a, s, r);
  const int warp = threadIdx.x >> 5;
  if (s.routed + shared_entries(a) == 0) {  // no expert of this part was picked
    for (int64_t i = blockIdx.x * THREADS + threadIdx.x; i < (int64_t)a.T * a.H; i += (int64_t)gridDim.x * THREADS)
      a.out[i] = a.shared_out != nullptr ? a.shared_out[i] : 0;
    return;
  }
  if (warp < WORKERS)
    work<W4>(a, s, smem_u32(smem));
  else if (warp == WORKERS)
    publish(a, s);
  else
    finish<W4>(a, s);
}

template <bool W4>
int launch(const FewArgs& a, cudaStream_t st) {
  const int nsm = device_sm_count();
  if (nsm <= 0) return MOE_ERR_CUDA;
  constexpr int smem = WORKERS * Fmt<W4>::STEPS * Fmt<W4>::STEP_BYTES;
  static_assert(smem + sizeof(Smem) + 1024 <= 232448 && smem >= (int)sizeof(Routing), "shared memory of a CTA");
  using Prep = void (*)(FewArgs);
  const Prep preps[4] = {prep_kernel<W4, 1>, prep_kernel<W4, 2>, prep_kernel<W4, 4>, prep_kernel<W4, 8>};
  static std::atomic<uint64_t> configured{0};  // a bit per device
  const int dev = current_device_index();
  if (dev < 0) return MOE_ERR_CUDA;
  if (!(configured.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    if (cudaFuncSetAttribute(few_kernel<W4>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return MOE_ERR_CUDA;
    // (an SM changes its split of L1 and shared memory only when it is empty: with its own split the prep kernel
    // would have to leave an SM before the other's CTA could be resident there)
    for (Prep p : preps)
      if (cudaFuncSetAttribute(p, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess) return MOE_ERR_CUDA;
    configured.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  }
  const int blocks = 1 + a.T + (a.logits == nullptr ? a.E * ((a.T + PREP_TOKENS - 1) / PREP_TOKENS) : 0);
  const Prep prep = preps[a.T == 1 ? 0 : a.T <= 2 ? 1 : a.T <= 4 ? 2 : 3];
  const int rc = launch_pdl(prep, dim3(blocks), dim3(PREP_THREADS), 0, st, a);
  if (rc != MOE_OK) return rc;
  return launch_pdl(few_kernel<W4>, dim3(nsm), dim3(THREADS), smem, st, a);
}

// Groups of a slice over `groups` groups of k, of a phase of `units` units a slice: 16 (64 KB of FP8 weights to a unit, 36 of
// NVFP4), and half or a quarter of that where it would leave the workers less than 1.5 units each.
int slice_groups(bool w4, int groups, int64_t units) {
  int want = 16;
  while (want > (w4 ? 4 : 2) && units * ((groups + want - 1) / want) < 3 * 152 * WORKERS / 2) want /= 2;
  const int slices = (groups + want - 1) / want, each = (groups + slices - 1) / slices;
  return w4 ? (each + 1) / 2 * 2 : each;
}

}  // namespace few_w4

// Workspace: offsets of the buffers; every counter is cleared by each call.
FewLayout few_w4_layout(bool w4, int T, int H, int I, int Is, int E, int k) {
  using namespace few_w4;
  FewLayout l = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += (bytes + 255) / 256 * 256;
    return was;
  };
  const size_t two = T > 8 ? 2 : 1, entries = std::min(two * E, (size_t)T * k) + (Is > 0 ? two : 0), slots = (size_t)T * k;
  const int deep = std::max(I, Is) / G;
  l.slice_groups[0] = slice_groups(w4, H / G, (int64_t)entries * (I / HALF));
  l.slice_groups[1] = slice_groups(w4, deep, (int64_t)entries * (H / ROWS));
  l.slices[0] = (H / G + l.slice_groups[0] - 1) / l.slice_groups[0];
  l.slices[1] = (deep + l.slice_groups[1] - 1) / l.slice_groups[1];
  l.groups_max = deep;
  // from an entry's last gate/up unit to its activations it takes some 7 us, 48 MB of weights
  const double gate_up = 2.0 * I * H * (w4 ? 9.0 / 16 : 1.0);
  l.lag = 1 << 20;
  l.n_ready = (int)entries;
  l.n_groups = (int)(entries * deep);
  l.n_columns = H / ROWS;
  l.n_counters = 64 + l.n_ready + l.n_groups + l.n_columns;
  l.y_slice = (slots + (Is > 0 ? T : 0)) * H;
  l.counters = take(4 * (size_t)l.n_counters);
  l.logits = take(4 * (size_t)T * E);
  l.x_values = take(T * (size_t)(H / G) * GROUP_BYTES);
  l.x_scales = take(4 * (size_t)T * (H / G));
  l.gu = take(4 * l.slices[0] * slots * 2 * I);
  l.act_values = take(slots * (I / G) * GROUP_BYTES);
  l.act_scales = take(4 * slots * (I / G));
  l.gu_shared = take(4 * l.slices[0] * (size_t)T * 2 * Is);
  l.act_values_shared = take((size_t)T * (Is / G) * GROUP_BYTES);
  l.act_scales_shared = take(4 * (size_t)T * (Is / G));
  l.Y = take(4 * l.slices[1] * l.y_slice);
  l.total = at;
  return l;
}

int few_w4_launch(bool w4, FewArgs& a, const FewLayout& l, void* ws, cudaStream_t st) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  auto floats = [&](size_t at) { return reinterpret_cast<float*>(base + at); };
  a.counters = reinterpret_cast<int*>(base + l.counters);
  a.ready = a.counters + 64;  // (on lines of their own behind the counters that units and tasks are drawn from)
  a.group_done = a.ready + l.n_ready;
  a.columns_done = a.group_done + l.n_groups;
  a.n_counters = l.n_counters;
  a.groups_max = l.groups_max;
  for (int i = 0; i < 2; ++i) {
    a.slices[i] = l.slices[i];
    a.slice_groups[i] = l.slice_groups[i];
  }
  a.y_slice = l.y_slice;
  a.lag = l.lag;
  a.logits_ws = floats(l.logits);
  a.x_made = base + l.x_values;
  a.x_scales_made = floats(l.x_scales);
  a.gu = floats(l.gu);
  a.act_codes = base + l.act_values;
  a.act_scales = floats(l.act_scales);
  a.gu_shared = floats(l.gu_shared);
  a.act_codes_shared = base + l.act_values_shared;
  a.act_scales_shared = floats(l.act_scales_shared);
  a.Y = floats(l.Y);
  return few_w4::launch<true>(a, st);
}

}  // namespace moe
