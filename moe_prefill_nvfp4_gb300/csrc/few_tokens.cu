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
//   prep     router logits (a CTA to an expert), the tokens' rows as records, counters to zero.
//   few      persistent, a CTA to an SM.  Each CTA routes the few tokens by itself (logits -> picks -> list of
//            the picked experts: the same in all CTAs), which is shorter than a launch, and then draws units
//            from a counter: first all experts' gate/up tiles, then all experts' down tiles.  A warp streams
//            the units' weights into a ring of shared memory, and because weights depend on no result, it runs
//            on into the down tiles while the activations that they need are still being made; only the small
//            activation records, which another warp fetches, wait for their expert.  Experts are drawn in the
//            same order in both halves, so an expert's activations are long finished when its down tiles come,
//            but for the last ones.
//
// A unit is a tile of 16 (FP8) or 32 (NVFP4) weight rows over all of k: 8 or 16 gate rows with their up rows, or
// as many down rows.  Eight warps share k (a group of 128 columns each), with the warp-level tensor-core
// products: the weight rows are the M operand, the expert's tokens the N operand (8 columns, or 16).  The 128 x
// 8 tiles that tcgen05 needs at least would be 1/16 rows that no token has, staged through tensor memory: at one
// to sixteen tokens there is nothing for its rate to do.  An epilogue warp adds the eight partial sums in order.
// The last of a group's 128 activations to be finished is the one that quantises them; the last of a tile's
// experts to be finished is the one that adds them up, in the order of the picks: no sum depends on who was last.
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
namespace few {

constexpr int G = 128;        // columns of a scale
constexpr int CHUNK = 8;      // groups of a stage: one to a warp
constexpr int MMA_WARPS = 8;
constexpr int MAX_EPI = 4;    // epilogue warps (and buffers of partial sums)
constexpr int THREADS = 32 * (2 + MMA_WARPS + MAX_EPI);
constexpr int MAX_STAGES = 16;
constexpr int MAX_T = MOE_FEW_MAX_TOKENS;
constexpr int MAX_SLOTS = MAX_T * 32;

// Shared-memory and record layouts.  A record is a token's (or an activation row's) part of a stage: 8 groups of
// 128 codes, then 8 scales; records lie 64 bytes past a multiple of 128 apart, so that the 16-byte loads of two
// neighbouring rows' four lanes take the 32 banks once.  The weights come as two blocks of ROWS / 2 rows by TMA:
// lines of 128 bytes (a group in FP8, two in NVFP4), the same of all rows in turn, with the 128-byte swizzle; the
// MMA's row g is row pi(g) of eight, so that neighbouring g differ in the swizzle's top bit, to the same effect.
// (A copy per row instead, 16 of 1 KB to a stage, took 2200 cycles a stage: bulk copies of a warp's lanes are
// issued one after another.  Two per stage.)
template <bool W4>
struct Fmt {
  static constexpr int ROWS = W4 ? 32 : 16;          // weight rows of a unit
  static constexpr int HALF = ROWS / 2;
  static constexpr int TILES = ROWS / 16;            // MMA tiles of a unit
  static constexpr int GROUP_BYTES = W4 ? 256 : 128; // of an activation row: FP16 or E4M3
  static constexpr int CODES = CHUNK * GROUP_BYTES;
  static constexpr int RECORD = CODES + 64;
  static constexpr int LINES = W4 ? 4 : 8;           // lines of a stage
  static constexpr int LINE_BYTES = HALF * 128;      // of one block's rows
  static constexpr int BLOCK_BYTES = LINES * LINE_BYTES;
  static constexpr int SCALES_AT = 2 * BLOCK_BYTES;  // NVFP4: 64 block scales to a row; FP8: 16 block scales (FP32)
  static constexpr int SCALES_BLOCK = HALF * 64;     // NVFP4: of one block's rows, with the 64-byte swizzle
  static constexpr int ACT_AT = SCALES_AT + (W4 ? 2 * SCALES_BLOCK : 64);
  static constexpr int LOADED = 2 * BLOCK_BYTES + (W4 ? 2 * SCALES_BLOCK : 0);
  static constexpr int PARTIAL = TILES * 512;        // a warp's partial sums per 8 tokens
  static constexpr int stage_bytes(int T) { return (ACT_AT + T * RECORD + 1023) / 1024 * 1024; }
};

// The row of eight that the MMA's row g is.
MOE_DEV int row_of(int g) { return (g >> 1) | ((g & 1) << 2); }

struct FewMaps {
  CUtensorMap w[4];  // FP8: gate/up, down; the shared expert's
};

MOE_DEV void load_3d(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
MOE_DEV void load_4d(uint32_t dst, const void* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

struct Entry {
  int expert;  // of the held ones; -1: the shared expert
  short m, first;
};

struct Smem {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], issued[MAX_STAGES];
  uint64_t part_full[MAX_EPI], part_empty[MAX_EPI];
  int4 info[MAX_STAGES];   // entry, tile, flags, groups
  int4 part_info[MAX_EPI]; // entry, tile, flags, warps with a part
  int routed, abort, issued_stages, filled_stages;
  float wts[MAX_SLOTS];
  short pos[MAX_SLOTS];              // row of slot (t, s), -1: of an expert held elsewhere
  uint8_t token[MAX_SLOTS + MAX_T];  // of row p
  Entry entry[MAX_SLOTS + 1];
};
// (only before the ring is used, in its place)
struct Routing {
  int32_t ids[MAX_SLOTS];
  uint32_t tokens[MOE_FEW_MAX_EXPERTS];  // bit t: token t has picked the expert
};

enum : int { DOWN = 1, FIRST = 2, LAST = 4, END = 8 };

MOE_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
MOE_DEV void copy4_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// arrives once this thread's copy4_async so far are done (an arrival of the barrier's own count)
MOE_DEV void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
MOE_DEV uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
MOE_DEV float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
MOE_DEV uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
MOE_DEV void sts_f32x4(uint32_t a, const float (&v)[4]) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}

// A whole warp's wait, with one outcome for all its lanes.
MOE_DEV bool warp_wait(uint64_t& bar, uint32_t parity, Smem& s, int* err) {
  return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity, &s.abort, err));
}

// D += A B, A 16 x 32 E4M3, B 32 x 8.  Lane (g = lane / 4, t = lane % 4): a0, a2 of row g, a1, a3 of row g + 8; b of
// column g; d0, d1 row g, columns 2t, 2t + 1; d2, d3 row g + 8.  Which k a register holds is free as long as A and B
// agree.
MOE_DEV void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with FP16 operands, A 16 x 16
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

// Group `grp` of a row, 4 consecutive columns to a lane, into the row's records, which lie `rows` records apart.
template <bool W4>
MOE_DEV void write_group(const float (&v)[4], uint8_t* first, int rows, int grp) {
  using F = Fmt<W4>;
  const int lane = threadIdx.x & 31;
  uint8_t* rec = first + (size_t)(grp / CHUNK) * rows * F::RECORD;
  uint8_t* codes = rec + (grp % CHUNK) * F::GROUP_BYTES;
  float scale;
  if constexpr (W4) {
    // a power of two that brings the group's largest finite magnitude to [2^14, 2^15): FP16 then holds BF16
    // numbers down to 2^-31 of it exactly, and FP32 ones to 2^-12 of their value; what is not finite stays so
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, abs_bits(v[i]) < 0x7F800000u ? abs_bits(v[i]) : 0u);
    m = __reduce_max_sync(0xffffffffu, m);
    const int ex = max((int)(m >> 23), 27);  // biased; at least 2^-100
    scale = __uint_as_float((uint32_t)(ex - 14) << 23);
    const float by = __uint_as_float((uint32_t)(254 - (ex - 14)) << 23);
    const __half2 lo = __floats2half2_rn(v[0] * by, v[1] * by), hi = __floats2half2_rn(v[2] * by, v[3] * by);
    // 8 columns to a piece of 16 bytes: lane t's pieces 4t .. 4t + 3 lie so that the four lanes' j-th are neighbours
    const int piece = lane >> 1;
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&lo);
    w.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(codes + ((piece & 3) * 4 + (piece >> 2)) * 16 + (lane & 1) * 8) = w;
  } else {
    const uint32_t m = __reduce_max_sync(
        0xffffffffu, max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3]))));
    float by;
    fp8_scale(m, scale, by);
    *reinterpret_cast<uint32_t*>(codes + lane * 4) = pack_e4m3x4(v[0] * by, v[1] * by, v[2] * by, v[3] * by);
  }
  if (lane == 0) reinterpret_cast<float*>(rec + F::CODES)[grp % CHUNK] = scale;
}

// ------------------------------------------------------------------------------------------------
// prep: block 0 clears the counters, blocks 1 .. T make the tokens' records, the others the router's logits

constexpr int PREP_THREADS = 256;

template <bool W4, int TT>
__global__ void __launch_bounds__(PREP_THREADS) prep_kernel(FewArgs a) {
  using F = Fmt<W4>;
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
    uint8_t* first = a.x_rec + (size_t)t * F::RECORD;
    const size_t apart = (size_t)a.T * F::RECORD;
    if (!W4 && a.rows_q != nullptr) {
      for (int p = threadIdx.x; p < a.H / 16; p += PREP_THREADS)
        *reinterpret_cast<uint4*>(first + (p / 64) * apart + (p % 64) * 16) =
            *reinterpret_cast<const uint4*>(a.rows_q + t * a.rows_ld + p * 16);
      for (int g = threadIdx.x; g < groups; g += PREP_THREADS)
        reinterpret_cast<float*>(first + (g / CHUNK) * apart + F::CODES)[g % CHUNK] =
            a.rows_s[t * a.rows_s_row + g * a.rows_s_grp];
    } else {
      for (int g = warp; g < groups; g += PREP_THREADS / 32) {
        const uint2 w = *reinterpret_cast<const uint2*>(a.x + (size_t)t * a.H + g * G + lane * 4);
        const float v[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
        write_group<W4>(v, first, a.T, g);
      }
    }
    return;
  }
  // one expert's logits of all tokens: its router row is read once, the tokens' rows come from the caches
  const int e = blockIdx.x - 1 - a.T;
  float acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.f;
  const uint4* w = reinterpret_cast<const uint4*>(a.w_router + (size_t)e * a.H);
  for (int i = threadIdx.x; i < a.H / 8; i += PREP_THREADS) {
    const uint4 wv = w[i];
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t >= a.T) break;
      const uint4 xv = reinterpret_cast<const uint4*>(a.x + (size_t)t * a.H)[i];
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
  if ((int)threadIdx.x < a.T) {
    float v = s_part[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < PREP_THREADS / 32; ++i) v += s_part[i][threadIdx.x];
    a.logits_ws[(size_t)threadIdx.x * a.E + e] = v;
  }
}

// ------------------------------------------------------------------------------------------------
// few: routing

MOE_DEV void route_rows(const FewArgs& a, Smem& s, Routing& r) {
  const float* logits = a.logits != nullptr ? a.logits : a.logits_ws;
  for (int t = threadIdx.x >> 5; t < a.T; t += THREADS / 32) {
    const float* row = logits + (size_t)t * a.E;
    int32_t* ids = r.ids + t * a.k;
    float* wts = s.wts + t * a.k;
    if (a.E <= 64)
      topk_row<2>(row, a.bias, a.E, a.k, a.renormalize, a.routed_scale, ids, wts, a.err);
    else if (a.E <= 256)
      topk_row<8>(row, a.bias, a.E, a.k, a.renormalize, a.routed_scale, ids, wts, a.err);
    else
      topk_row<16>(row, a.bias, a.E, a.k, a.renormalize, a.routed_scale, ids, wts, a.err);
  }
}

// The list of the picked experts that are held here, in expert order, and their rows, in token order: row p of
// an entry is row p of the activation records and of Y.  A shared expert is entry 0, with rows T k .. T k + T - 1.
template <bool W4>
MOE_DEV void make_entries(const FewArgs& a, Smem& s, Routing& r) {
  const int slots = a.T * a.k, tid = threadIdx.x, lane = tid & 31;
  for (int e = tid; e < a.E; e += THREADS) r.tokens[e] = 0;
  __syncthreads();
  route_rows(a, s, r);
  __syncthreads();
  for (int i = tid; i < slots; i += THREADS) {
    const int e = r.ids[i];
    s.pos[i] = -1;
    const bool held = W4 ? a.w4[0].packed[e] != nullptr && a.w4[1].packed[e] != nullptr
                         : e >= a.first && e < a.first + a.count;
    if (held) atomicOr(&r.tokens[e], 1u << (i / a.k));
  }
  __syncthreads();
  const int sh = a.Is > 0;
  if (tid < 32) {
    int n = sh, p = 0;
    for (int e0 = 0; e0 < a.count; e0 += 32) {
      const uint32_t mine = e0 + lane < a.count ? r.tokens[a.first + e0 + lane] : 0u;
      const int m = __popc(mine);
      int rows = m;  // inclusive prefix over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, rows, o);
        if (lane >= o) rows += v;
      }
      const uint32_t used = __ballot_sync(0xffffffffu, m > 0);
      if (m > 0) {
        const int first = p + rows - m;
        s.entry[n + __popc(used & ((1u << lane) - 1))] = Entry{e0 + lane, (short)m, (short)first};
        int q = first;
        for (uint32_t b = mine; b != 0; b &= b - 1) s.token[q++] = (uint8_t)(__ffs(b) - 1);
      }
      n += __popc(used);
      p += __shfl_sync(0xffffffffu, rows, 31);
    }
    if (lane == 0) {
      s.routed = n - sh;
      if (sh) s.entry[0] = Entry{-1, (short)a.T, (short)slots};
    }
    if (sh && lane < a.T) s.token[slots + lane] = (uint8_t)lane;
  }
  __syncthreads();
  // where each slot's row is: found in its expert's entry
  for (int i = tid; i < s.routed; i += THREADS) {
    const Entry en = s.entry[sh + i];
    for (int j = 0; j < en.m; ++j) {
      const int t = s.token[en.first + j];
      for (int c = 0; c < a.k; ++c)
        if (r.ids[t * a.k + c] == a.first + en.expert) s.pos[t * a.k + c] = (short)(en.first + j);
    }
  }
  __syncthreads();
}

struct Unit {
  int entry, tile;
  bool down;
};
template <bool W4>
struct Units {
  int shared, gate_up, total, sh, per_gu, per_down;
  MOE_DEV Units(const FewArgs& a, int routed) {
    sh = a.Is > 0;
    per_gu = a.I / Fmt<W4>::HALF;
    per_down = a.H / Fmt<W4>::ROWS;
    shared = sh ? a.Is / Fmt<W4>::HALF : 0;
    gate_up = shared + routed * per_gu;
    total = gate_up + (routed + sh) * per_down;
  }
  MOE_DEV Unit at(int u) const {
    if (u < shared) return Unit{0, u, false};
    if (u < gate_up) {
      const int v = u - shared;
      return Unit{sh + v / per_gu, v % per_gu, false};
    }
    const int v = u - gate_up;
    return Unit{v / per_down, v % per_down, true};
  }
};

// ------------------------------------------------------------------------------------------------
// few: the roles

// Streams the weights of the units that this CTA draws.
template <bool W4>
MOE_DEV void load_weights(const FewArgs& a, const FewMaps& maps, Smem& s, uint32_t ring, int stages) {
  using F = Fmt<W4>;
  const int lane = threadIdx.x & 31, stage_bytes = F::stage_bytes(a.T);
  const Units<W4> units(a, s.routed);
  int it = 0, slot = 0, phase = 0;
  auto draw = [&]() { return lane == 0 ? atomicAdd(a.counters, 1) : 0; };
  int next = draw();
  for (;;) {
    const int u = __shfl_sync(0xffffffffu, next, 0);
    if (u >= units.total) break;
    next = draw();  // (its answer is there when this unit's copies are on their way)
    const Unit un = units.at(u);
    const Entry en = s.entry[un.entry];
    const bool is_shared = en.expert < 0;
    const int inter = is_shared ? a.Is : a.I;
    const int groups = (un.down ? inter : a.H) / G;
    // the two blocks' first rows
    const int row0 = un.down ? un.tile * F::ROWS : un.tile * F::HALF;
    const int row1 = un.down ? row0 + F::HALF : row0 + inter;
    const CUtensorMap* map;
    const float* scales = nullptr;
    if constexpr (W4) {
      map = a.w4[un.down].maps + 2 * (a.first + en.expert);
    } else {
      map = &maps.w[(is_shared ? 2 : 0) + un.down];
      const FewFp8Weight& w = is_shared ? a.w8s[un.down] : a.w8[un.down];
      const size_t blocks = (un.down ? a.H : 2 * inter) / G;
      // (lanes 0-7: a group each of the first block's scales, 8-15: of the second's)
      scales = w.s + ((is_shared ? 0 : en.expert) * blocks + (lane < 8 ? row0 : row1) / G) * groups + (lane & 7);
    }
    for (int g0 = 0; g0 < groups; g0 += CHUNK) {
      const int n = min(CHUNK, groups - g0);
      if (!warp_wait(s.empty[slot], phase ^ 1, s, a.err)) goto out;
      const uint32_t full = smem_u32(&s.full[slot]), at = ring + slot * stage_bytes;
      if (lane == 0) {
        s.info[slot] = make_int4(un.entry, un.tile, (un.down ? DOWN : 0) | (g0 == 0 ? FIRST : 0) | (g0 + n == groups ? LAST : 0), n);
        mbar_arrive_expect_tx(full, F::LOADED);  // (lines past k come as zeros)
        if constexpr (W4) {
          load_3d(at, map, 0, row0, g0 / 2, full);
          load_3d(at + F::BLOCK_BYTES, map, 0, row1, g0 / 2, full);
          tma_load_2d(at + F::SCALES_AT, map + 1, g0 * 8, row0, full);
          tma_load_2d(at + F::SCALES_AT + F::SCALES_BLOCK, map + 1, g0 * 8, row1, full);
        } else {
          const int e = is_shared ? 0 : en.expert;
          load_4d(at, map, 0, row0, g0, e, full);
          load_4d(at + F::BLOCK_BYTES, map, 0, row1, g0, e, full);
        }
        mbar_arrive(smem_u32(&s.issued[slot]));
      }
      if constexpr (!W4) {
        if (lane < 16 && (lane & 7) < n) copy4_async(at + F::SCALES_AT + lane * 4, scales + g0);
        copies_arrive(full);
      }
      ++it;
      if (++slot == stages) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
  if (warp_wait(s.empty[slot], phase ^ 1, s, a.err)) {
    const uint32_t full = smem_u32(&s.full[slot]);
    if (lane == 0) {
      s.info[slot] = make_int4(0, 0, END, 0);
      mbar_arrive(full);
      mbar_arrive(smem_u32(&s.issued[slot]));
    }
    if constexpr (!W4) copies_arrive(full);
    ++it;
  }
out:
  if (lane == 0) s.issued_stages = it;
}

// Fetches the activation records of the same units, once they are finished.
template <bool W4>
MOE_DEV void load_records(const FewArgs& a, Smem& s, uint32_t ring, int stages) {
  using F = Fmt<W4>;
  const int lane = threadIdx.x & 31, stage_bytes = F::stage_bytes(a.T);
  int it = 0, slot = 0, phase = 0, ready = -1, chunk = 0;
  fence_proxy_async_global();  // (the tokens' records, stored by the launch before)
  for (;;) {
    if (!warp_wait(s.issued[slot], phase, s, a.err)) break;
    const int4 in = s.info[slot];
    const uint32_t full = smem_u32(&s.full[slot]);
    if (in.z & END) {
      if (lane == 0) mbar_arrive(full);
      ++it;
      break;
    }
    if (in.z & FIRST) chunk = 0;
    const Entry en = s.entry[in.x];
    const uint32_t to = ring + slot * stage_bytes + F::ACT_AT;
    if (in.z & DOWN) {
      const int inter = en.expert < 0 ? a.Is : a.I;
      if (ready != in.x) {
        int ok = 1;
        if (lane == 0) ok = wait_counter_geq(a.ready + in.x, inter / G, &s.abort, a.err);
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        fence_proxy_async_global();
        ready = in.x;
      }
    }
    if (lane == 0) mbar_arrive_expect_tx(full, en.m * F::RECORD);
    __syncwarp();
    // an expert's activations lie one after another, and so do the rows of an expert that has all tokens
    if ((in.z & DOWN) || en.m == a.T) {
      const uint8_t* src = !(in.z & DOWN)  ? a.x_rec + (size_t)(chunk * a.T) * F::RECORD
                           : en.expert < 0 ? a.act_rec_shared + (size_t)(chunk * a.T) * F::RECORD
                                           : a.act_rec + (size_t)(chunk * a.T * a.k + en.first) * F::RECORD;
      if (lane == 0) bulk_load(to, src, en.m * F::RECORD, full);
    } else if (lane < en.m) {
      bulk_load(to + lane * F::RECORD, a.x_rec + (size_t)(chunk * a.T + s.token[en.first + lane]) * F::RECORD, F::RECORD, full);
    }
    ++chunk;
    ++it;
    if (++slot == stages) {
      slot = 0;
      phase ^= 1;
    }
  }
  if (lane == 0) s.filled_stages = it;
}

// This warp's group of a stage: acc += scale * (codes' products), for NT columns of 8 tokens.
template <bool W4, int NT>
MOE_DEV void group_product(uint32_t at, int warp, int m, bool down, float (&acc)[Fmt<W4>::TILES][2][4]) {
  using F = Fmt<W4>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t b_at[NT];
  float sa[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // (columns past the expert's last token repeat it: their sums are not stored)
    b_at[n] = at + F::ACT_AT + min(n * 8 + g, m - 1) * F::RECORD + warp * F::GROUP_BYTES + t * 16;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      sa[n][c] = lds_f32(at + F::ACT_AT + min(n * 8 + 2 * t + c, m - 1) * F::RECORD + F::CODES + warp * 4);
  }
  const int rg = row_of(g);
  float tmp[F::TILES][NT][4];
#pragma unroll
  for (int i = 0; i < F::TILES; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) tmp[i][n][0] = tmp[i][n][1] = tmp[i][n][2] = tmp[i][n][3] = 0.f;
  if constexpr (W4) {
    // 32 consecutive k to a lane (16 bytes of each row), 8 to a word: two MMAs
    uint4 p[4];
    uint32_t sc[4][2];
    // (tile i / 2's rows g, then its rows g + 8: gate and up, or the two halves of one block)
    const uint32_t line = at + (warp >> 1) * F::LINE_BYTES + rg * 128 + ((((warp & 1) * 4 + t) ^ rg) << 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int block = down ? i >> 1 : i & 1, eight = down ? i & 1 : i >> 1;
      p[i] = lds128(line + block * F::BLOCK_BYTES + eight * 1024);
      uint32_t both, unused;
      e4m3x4_to_f16x2(lds_u16(at + F::SCALES_AT + block * F::SCALES_BLOCK + (eight * 8 + rg) * 64 +
                              (((warp >> 1) ^ (rg >> 1)) << 4) + (warp & 1) * 8 + t * 2),
                      both, unused);
      sc[i][0] = prmt(both, both, 0x1010);
      sc[i][1] = prmt(both, both, 0x3232);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n] = lds128(b_at[n] + j * 64);
      uint32_t h[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e2m1x8_to_f16x2(j == 0 ? p[i].x : j == 1 ? p[i].y : j == 2 ? p[i].z : p[i].w, h[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) h[i][q] = mul_f16x2(h[i][q], sc[i][j >> 1]);  // exact: at most 6 bits
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(tmp[i][n], h[2 * i][0], h[2 * i + 1][0], h[2 * i][1], h[2 * i + 1][1], b[n].x, b[n].y);
          mma_f16(tmp[i][n], h[2 * i][2], h[2 * i + 1][2], h[2 * i][3], h[2 * i + 1][3], b[n].z, b[n].w);
        }
    }
#pragma unroll
    for (int i = 0; i < F::TILES; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][n][c] = __fmaf_rn(tmp[i][n][c], sa[n][c & 1], acc[i][n][c]);
  } else {
    const uint32_t line = at + warp * F::LINE_BYTES + rg * 128;
    const float sw[2] = {lds_f32(at + F::SCALES_AT + warp * 4), lds_f32(at + F::SCALES_AT + 32 + warp * 4)};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t piece = line + (((j * 4 + t) ^ rg) << 4);
      const uint4 lo = lds128(piece), hi = lds128(piece + F::BLOCK_BYTES);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = lds128(b_at[n] + j * 64);
        mma_e4m3(tmp[0][n], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
        mma_e4m3(tmp[0][n], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[0][n][c] = __fmaf_rn(tmp[0][n][c], sa[n][c & 1] * sw[c >> 1], acc[0][n][c]);
  }
}

template <bool W4>
MOE_DEV void multiply(const FewArgs& a, Smem& s, uint32_t ring, uint32_t parts, int stages, int nbuf) {
  using F = Fmt<W4>;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 2, stage_bytes = F::stage_bytes(a.T);
  const int nt_max = a.T > 8 ? 2 : 1;
  int slot = 0, phase = 0, buf = 0, buf_phase = 0, parts_of = 0;
  float acc[F::TILES][2][4];
  auto hand_over = [&](const int4& in, int flags) {
    if (!warp_wait(s.part_empty[buf], buf_phase ^ 1, s, a.err)) return false;
    if (!(flags & END) && warp < parts_of) {
      const int nt = s.entry[in.x].m > 8 ? 2 : 1;
      const uint32_t to = parts + (uint32_t)((buf * MMA_WARPS + warp) * nt_max) * F::PARTIAL + lane * 16;
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (n < nt)
#pragma unroll
          for (int i = 0; i < F::TILES; ++i) sts_f32x4(to + (n * F::TILES + i) * 512, acc[i][n]);
    }
    if (warp == 0 && lane == 0) s.part_info[buf] = make_int4(in.x, in.y, flags, parts_of);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.part_full[buf]));
    if (++buf == nbuf) {
      buf = 0;
      buf_phase ^= 1;
    }
    return true;
  };
  for (;;) {
    if (!warp_wait(s.full[slot], phase, s, a.err)) return;
    const int4 in = s.info[slot];
    if (in.z & END) {
      for (int i = 0; i < nbuf; ++i)
        if (!hand_over(in, END)) return;
      return;
    }
    if (in.z & FIRST) {
      parts_of = in.w;
#pragma unroll
      for (int i = 0; i < F::TILES; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
    }
    if (warp < in.w) {
      const int m = s.entry[in.x].m;
      const uint32_t at = ring + slot * stage_bytes;
      if (m <= 8)
        group_product<W4, 1>(at, warp, m, in.z & DOWN, acc);
      else
        group_product<W4, 2>(at, warp, m, in.z & DOWN, acc);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.empty[slot]));
    if (++slot == stages) {
      slot = 0;
      phase ^= 1;
    }
    if ((in.z & LAST) && !hand_over(in, in.z)) return;
  }
}

// Adds the warps' parts of a unit and passes the sums on: gate and up to an activation (and the group's
// quantiser), down to Y (and the tile's weighted sum).
template <bool W4>
MOE_DEV void finish(const FewArgs& a, Smem& s, uint32_t parts, int nbuf) {
  using F = Fmt<W4>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int buf = (threadIdx.x >> 5) - 2 - MMA_WARPS;
  if (buf >= nbuf) return;
  const int nt_max = a.T > 8 ? 2 : 1, slots = a.T * a.k;
  for (int phase = 0;; phase ^= 1) {
    if (!warp_wait(s.part_full[buf], phase, s, a.err)) return;
    const int4 in = s.part_info[buf];
    if (in.z & END) return;
    const Entry en = s.entry[in.x];
    const int nt = en.m > 8 ? 2 : 1;
    float sum[F::TILES][2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
      if (n < nt)
#pragma unroll
        for (int i = 0; i < F::TILES; ++i) {
          const uint32_t from = parts + (uint32_t)(buf * MMA_WARPS * nt_max) * F::PARTIAL + (n * F::TILES + i) * 512 + lane * 16;
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          for (int w = 0; w < in.w; ++w) {
            const uint4 p = lds128(from + (uint32_t)(w * nt_max) * F::PARTIAL);
            v[0] += __uint_as_float(p.x);
            v[1] += __uint_as_float(p.y);
            v[2] += __uint_as_float(p.z);
            v[3] += __uint_as_float(p.w);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) sum[i][n][c] = v[c];
        }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.part_empty[buf]));
    const bool is_shared = en.expert < 0;
    if constexpr (W4) {
      const float s2 = a.w4[(in.z & DOWN) ? 1 : 0].scale2[a.first + en.expert];
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (n < nt)
#pragma unroll
          for (int i = 0; i < F::TILES; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[i][n][c] *= s2;
    }
    if (!(in.z & DOWN)) {
      const int inter = is_shared ? a.Is : a.I, j0 = in.y * F::HALF;
      float* act = is_shared ? a.act_shared : a.act + (size_t)en.first * a.I;
      const float limit = is_shared ? a.shared_limit : a.limit;
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (n < nt)
#pragma unroll
          for (int i = 0; i < F::TILES; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = n * 8 + 2 * t + c;
              if (col < en.m) act[(size_t)col * inter + j0 + i * 8 + row_of(g)] = swiglu_keep_nan<false>(sum[i][n][c], sum[i][n][2 + c], limit);
            }
      const int grp = j0 / G;
      __syncwarp();
      int last = 0;
      if (lane == 0) {
        __threadfence();
        last = atomicAdd(a.group_done + in.x * a.groups_max + grp, 1) == G / F::HALF - 1;
        __threadfence();
      }
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      __syncwarp();
      uint8_t* rec = is_shared ? a.act_rec_shared : a.act_rec + (size_t)en.first * F::RECORD;
      const int apart = is_shared ? a.T : slots;
      for (int r0 = 0; r0 < en.m; r0 += 4) {
        float4 v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (r0 + r < en.m) v[r] = __ldcg(reinterpret_cast<const float4*>(act + (size_t)(r0 + r) * inter + grp * G) + lane);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (r0 + r < en.m) {
            const float f[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
            write_group<W4>(f, rec + (size_t)(r0 + r) * F::RECORD, apart, grp);
          }
      }
      __syncwarp();
      if (lane == 0) {
        __threadfence();
        counter_add_release(a.ready + in.x, 1);
      }
    } else {
      const int h0 = in.y * F::ROWS;
      float* y = a.Y + (size_t)en.first * a.H + h0;
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (n < nt)
#pragma unroll
          for (int i = 0; i < F::TILES; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int col = n * 8 + 2 * t + (c & 1);
              if (col < en.m) y[(size_t)col * a.H + i * 16 + row_of(g) + 8 * (c >> 1)] = sum[i][n][c];
            }
      __syncwarp();
      const int entries = s.routed + (a.Is > 0);
      int last = 0;
      if (lane == 0) {
        __threadfence();
        last = atomicAdd(a.tile_done + in.y, 1) == entries - 1;
        __threadfence();
      }
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      __syncwarp();
      const int h = h0 + (lane & (F::ROWS - 1));
      for (int tok = lane / F::ROWS; tok < a.T; tok += 32 / F::ROWS) {
        float v = 0.f;
        for (int c0 = 0; c0 < a.k; c0 += 8) {
          float yv[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int p = c0 + c < a.k ? s.pos[tok * a.k + c0 + c] : -1;
            yv[c] = p >= 0 ? __ldcg(a.Y + (size_t)p * a.H + h) : 0.f;
          }
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c0 + c < a.k && s.pos[tok * a.k + c0 + c] >= 0) v = __fmaf_rn(s.wts[tok * a.k + c0 + c], yv[c], v);
        }
        if (a.Is > 0) v += __ldcg(a.Y + (size_t)(slots + tok) * a.H + h);
        if (a.shared_out != nullptr) v += __bfloat162float(__ushort_as_bfloat16(a.shared_out[(size_t)tok * a.H + h]));
        a.out[(size_t)tok * a.H + h] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
      }
    }
  }
}

template <bool W4>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ FewArgs a, const __grid_constant__ FewMaps maps, int stages,
                                                          int nbuf) {
  using F = Fmt<W4>;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t ring = (smem_u32(smem) + 1023) / 1024 * 1024;  // (the swizzle goes by address bits)
  uint8_t* behind = smem + (ring - smem_u32(smem)) + stages * F::stage_bytes(a.T);
  const uint32_t parts = smem_u32(behind);
  Smem& s = *reinterpret_cast<Smem*>(behind + nbuf * MMA_WARPS * (a.T > 8 ? 2 : 1) * F::PARTIAL);
  Routing& r = *reinterpret_cast<Routing*>(smem + (ring - smem_u32(smem)));
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(smem_u32(&s.full[i]), W4 ? 2 : 2 + 32);  // weights, records (and the scales' copies)
      mbar_init(smem_u32(&s.empty[i]), MMA_WARPS);
      mbar_init(smem_u32(&s.issued[i]), 1);
    }
    for (int i = 0; i < nbuf; ++i) {
      mbar_init(smem_u32(&s.part_full[i]), MMA_WARPS);
      mbar_init(smem_u32(&s.part_empty[i]), 1);
    }
    s.abort = 0;
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  make_entries<W4>(a, s, r);  // (a barrier on every path)
  const int warp = threadIdx.x >> 5;
  if (s.routed + (a.Is > 0) == 0) {  // no expert of this part was picked
    for (int64_t i = blockIdx.x * THREADS + threadIdx.x; i < (int64_t)a.T * a.H; i += (int64_t)gridDim.x * THREADS)
      a.out[i] = a.shared_out != nullptr ? a.shared_out[i] : 0;
    return;
  }
  fence_proxy_async_shared();  // (the ring's first bytes were the routing's)
  __syncthreads();
  if (warp == 0)
    load_weights<W4>(a, maps, s, ring, stages);
  else if (warp == 1)
    load_records<W4>(a, s, ring, stages);
  else if (warp < 2 + MMA_WARPS)
    multiply<W4>(a, s, ring, parts, stages, nbuf);
  else
    finish<W4>(a, s, parts, nbuf);
  __syncthreads();
  // after a wait that ran out: no copy may still be on its way into a CTA that is gone
  if (s.abort && threadIdx.x == 0) {
    for (int it = s.filled_stages; it < s.issued_stages; ++it) mbar_arrive(smem_u32(&s.full[it % stages]));
    for (int it = max(0, s.issued_stages - stages); it < s.issued_stages; ++it)
      mbar_wait_drain(smem_u32(&s.full[it % stages]), (it / stages) & 1);
  }
}

// An FP8 weight as lines of 128 columns: line of a row, row, line's place in the row, expert; 8 rows by 8 lines.
int weight_map(CUtensorMap* map, const FewFp8Weight& w, int N, int K, int count) {
  const cuuint64_t dims[4] = {128, (cuuint64_t)N, (cuuint64_t)(K / 128), (cuuint64_t)count};
  const cuuint64_t strides[3] = {(cuuint64_t)w.ld, 128, (cuuint64_t)(count > 1 ? w.expert_stride : w.ld * (int64_t)N)};
  const cuuint32_t box[4] = {128, 8, 8, 1}, one[4] = {1, 1, 1, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(w.q), dims, strides, box, one,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool W4>
int launch(const FewArgs& a, cudaStream_t st) {
  using F = Fmt<W4>;
  const int nsm = device_sm_count();
  if (nsm <= 0) return MOE_ERR_CUDA;
  // (the partial sums of 16 tokens over 32 rows are 16 KB to a buffer: two of them then)
  const int nbuf = W4 && a.T > 8 ? 2 : MAX_EPI;
  constexpr int kSmem = 232448 - 1024;
  const int fixed = (int)sizeof(Smem) + nbuf * MMA_WARPS * (a.T > 8 ? 2 : 1) * F::PARTIAL;
  const int stages = std::min(MAX_STAGES, (kSmem - fixed) / F::stage_bytes(a.T));
  const int smem = 1024 + fixed + stages * F::stage_bytes(a.T);
  static_assert(F::stage_bytes(1) * 2 >= (int)sizeof(Routing), "the routing has its arrays in the ring");
  static std::atomic<uint64_t> configured{0};  // a bit per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (!(configured.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    if (cudaFuncSetAttribute(few_kernel<W4>, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kSmem) != cudaSuccess)
      return MOE_ERR_CUDA;
    configured.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  }
  FewMaps maps = {};
  if constexpr (!W4) {
    int rc = weight_map(&maps.w[0], a.w8[0], 2 * a.I, a.H, a.count);
    if (rc == MOE_OK) rc = weight_map(&maps.w[1], a.w8[1], a.H, a.I, a.count);
    if (rc == MOE_OK && a.Is > 0) rc = weight_map(&maps.w[2], a.w8s[0], 2 * a.Is, a.H, 1);
    if (rc == MOE_OK && a.Is > 0) rc = weight_map(&maps.w[3], a.w8s[1], a.H, a.Is, 1);
    if (rc != MOE_OK) return rc;
  }
  const int blocks = 1 + a.T + (a.logits == nullptr ? a.E : 0);
  auto prep = a.T == 1 ? prep_kernel<W4, 1> : a.T <= 2 ? prep_kernel<W4, 2> : a.T <= 4 ? prep_kernel<W4, 4>
                       : a.T <= 8 ? prep_kernel<W4, 8> : prep_kernel<W4, 16>;
  const int rc = launch_pdl(prep, dim3(blocks), dim3(PREP_THREADS), 0, st, a);
  if (rc != MOE_OK) return rc;
  return launch_pdl(few_kernel<W4>, dim3(nsm), dim3(THREADS), smem, st, a, maps, stages, nbuf);
}

}  // namespace few

// Workspace: offsets of the buffers; every counter is cleared by each call.
FewLayout few_layout(bool w4, int T, int H, int I, int Is, int E, int k) {
  FewLayout l = {};
  const size_t record = w4 ? few::Fmt<true>::RECORD : few::Fmt<false>::RECORD;
  const size_t rows = w4 ? few::Fmt<true>::ROWS : few::Fmt<false>::ROWS;
  auto chunks = [](int n) { return (size_t)(n / few::G + few::CHUNK - 1) / few::CHUNK; };
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += (bytes + 255) / 256 * 256;
    return was;
  };
  const size_t entries = (size_t)std::min(E, T * k) + (Is > 0);
  l.groups_max = std::max(I, Is) / few::G;
  l.n_ready = (int)entries;
  l.n_groups = (int)(entries * l.groups_max);
  l.n_tiles = (int)(H / rows);
  l.n_counters = 32 + l.n_ready + l.n_groups + l.n_tiles;
  l.counters = take(4 * (size_t)l.n_counters);
  l.logits = take(4 * (size_t)T * E);
  l.x_rec = take(T * chunks(H) * record);
  l.act = take(4 * (size_t)T * k * I);
  l.act_shared = take(4 * (size_t)T * Is);
  l.act_rec = take((size_t)T * k * chunks(I) * record);
  l.act_rec_shared = take(T * chunks(Is) * record);
  l.Y = take(4 * ((size_t)T * k + (Is > 0 ? T : 0)) * H);
  l.total = at;
  return l;
}

int few_launch(bool w4, FewArgs& a, const FewLayout& l, void* ws, cudaStream_t st) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.counters = reinterpret_cast<int*>(base + l.counters);
  a.ready = a.counters + 32;  // (on lines of their own behind the counter that units are drawn from)
  a.group_done = a.ready + l.n_ready;
  a.tile_done = a.group_done + l.n_groups;
  a.n_counters = l.n_counters;
  a.groups_max = l.groups_max;
  a.logits_ws = reinterpret_cast<float*>(base + l.logits);
  a.x_rec = base + l.x_rec;
  a.act = reinterpret_cast<float*>(base + l.act);
  a.act_shared = reinterpret_cast<float*>(base + l.act_shared);
  a.act_rec = base + l.act_rec;
  a.act_rec_shared = base + l.act_rec_shared;
  a.Y = reinterpret_cast<float*>(base + l.Y);
  return w4 ? few::launch<true>(a, st) : few::launch<false>(a, st);
}

}  // namespace moe
