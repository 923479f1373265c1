// few.cuh -- a whole layer of routed experts (and a shared one) for at most 16 tokens, in two launches:
//
//   out[t] = sum_s wts[t, s] * W_dn[e] act(W_gu[e] x[t])  (+ shared),  e = ids[t, s],
//   act = silu(min(g, L)) * clamp(u, -L, L)
//
// Bound by the weights' bytes: of each expert that a token has picked, once.  So everything else is kept out of
// their way:
//   prep  router logits (a CTA to an expert and four tokens), the tokens' rows in the form of the products' operand,
//         counters to zero.
//   few   persistent, two CTAs to an SM.  Each CTA routes the few tokens by itself (logits -> picks -> list of the
//         picked experts: the same in all CTAs), which is shorter than a launch.  Then it draws units from a counter --
//         256 weight rows (128 gate rows with their up rows, or 256 down rows) over a slice of k -- and streams their
//         weights through its stages without a pause between units.  Because weights depend on no result, the stream
//         runs on into down units while the activations that those need are still being made; only the loader of the
//         activations waits.
//
// The weight rows are the tensor-core MMA's M operand, the expert's tokens, 16 at most, its N operand; a k block makes
// one accumulator, which the epilogue scales and adds to FP32 registers.  A unit's sums go to memory by slices.  A warp
// that waits for the last one that an activation block needs adds the slices in order, and makes the activations
// and brings them into the operand's form; another such task adds up slices and experts of 32 columns of the result.
// No sum depends on who was last.
//
// Kernel time (160 experts, top-8, 5120 x 1536, in graphs of calls with other tokens): one token 46 us in FP8 and 40 in
// NVFP4, 16 tokens 316 and 202; the picked weights' bytes take 28 and 16, 311 and 175 us.  What is above that is latency:
// 4 us of logits, 4 of routing, 5 to the first stages (their code comes from L2 too), 4 between the last gate/up sums and
// the down products, 5 from the last sums to the result.
//
// Units and tasks are drawn behind all that they need, so whichever CTAs are running make progress, also beside another
// call's kernel that holds a part of the SMs.  Every wait is bounded (FewArgs::wait_ns, MOE_DEVERR_TIMEOUT).
//
// What differs between the weights' formats is in a class F:
//   KB                       columns of a k block (of the weights' 128 bytes, one swizzle row)
//   STAGE                    bytes of a stage: 256 weight rows of 128 bytes, then what goes with them
//   TMEM_COLS, accumulators(most)   tensor memory, and the accumulators in it for units of that many tokens at most
//   WEIGHT_ARRIVALS, FULL_ARRIVALS   arrivals that make a stage full: the weights', and with the rows'
//   Maps, held(a, e)         tensor maps by value, whether expert e is here
//   Weights, Rows            the loads of a unit's k blocks: the weights, and the rows with their scales
//   multiply, add            a stage's MMAs, an accumulator's scaling and addition
//   output_scale(a, expert)  factor of a unit's sums
//   LANE, write_block        a block of KB columns of a row, LANE to a lane, into the operand's form
#pragma once

#include <algorithm>
#include <atomic>

#include "few.h"
#include "fp8_mma.cuh"
#include "internal.h"
#include "topk.cuh"

namespace moe {
namespace few {

using namespace f8;

constexpr int NT = 16;             // tokens of a unit
constexpr int NS = 2;              // stages: 128 KB of an SM on their way (a third: 57 us for one token instead of 53)
constexpr int ND = 8;              // accumulators, at most
constexpr int NF = 16;             // k blocks whose scales are held, more than accumulators and stages together
constexpr int F_SLOT = NT + 4;     // the rows' scales, then the weight's
constexpr int DRAWN = 8;           // units that a CTA has drawn and not finished
// warps: 0 draws and loads weights, 1 issues MMAs, 2-5 epilogue, 6 loads activations, 7 publishes, 8 and 9 finish
constexpr int WARPS = 10;
constexpr int THREADS = 32 * WARPS;
constexpr int PER_SM = 2;
constexpr int MAX_T = MOE_FEW_MAX_TOKENS;
constexpr int MAX_SLOTS = MAX_T * 32;
static_assert(NF >= ND + NS && MAX_T <= NT, "");

struct Entry {
  int expert;  // of the held ones; -1: the shared expert
  short m, first;
};
struct Unit {
  int entry, expert, m, first;  // its list entry, with its expert and rows
  int place, slice;             // of its weight rows among the entry's; of k
  int kb0, kb1;                 // its k blocks
  int flags;                    // DOWN, SHARED, END
};
enum : int { DOWN = 1, SHARED = 2, END = 4 };

struct Smem {
  uint64_t full[NS], empty[NS], d_full[ND], d_empty[ND], drawn[DRAWN], spent[DRAWN], stored[DRAWN], drain;
  Unit unit[DRAWN];
  alignas(16) float scales[NF][F_SLOT];
  uint32_t tmem;
  int routed, rows, most, abort;     // picked experts, their rows, tokens of one at most
  int weights_issued, rows_issued;   // k blocks whose weights and whose rows were loaded, once their loaders have ended
  float wts[MAX_SLOTS];
  short pos[MAX_SLOTS];              // row of slot (t, s), -1: of an expert held elsewhere
  uint8_t token[MAX_SLOTS + MAX_T];  // of row p
  short entry_of[MAX_SLOTS];         // of row p, not of a shared expert's
  Entry entry[MAX_SLOTS + 1];
};
static_assert(offsetof(Smem, scales) % 16 == 0 && F_SLOT % 4 == 0, "read by 16 bytes");
// (only before the stages are used, in their place)
struct Routing {
  int32_t ids[MAX_SLOTS];
  uint32_t tokens[MOE_FEW_MAX_EXPERTS];  // bit t: token t has picked the expert
  short first[MOE_FEW_MAX_EXPERTS];      // its first row
  int sums[MOE_FEW_MAX_EXPERTS / 32];    // of 32 experts each: rows, experts << 16
  bool held[MOE_FEW_MAX_EXPERTS];        // the expert is here
};

// The weights are read once and are more than L2 holds: as the first to be evicted they leave it to what every layer
// needs again, above all to this kernel's instructions (one token 50 -> 45 us in FP8, 16 tokens 329 -> 317).
MOE_DEV uint64_t streaming_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

MOE_DEV uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

MOE_DEV bool warp_wait(uint64_t& bar, uint32_t parity, Smem& s, const FewArgs& a) {
  return mbar_wait_warp(smem_u32(&bar), parity, &s.abort, a.err, a.wait_ns);
}

// Waits for a count of what other warps have stored and published (a poll is a round trip to L2).
MOE_DEV bool wait_count(const int* count, int need, Smem& s, const FewArgs& a) {
  int ok = 1;
  if (lane_id() == 0) {
    uint64_t t0 = 0;
    for (int n = 1;; ++n) {
      int v;
      asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
      if (v >= need) break;
      ok = !*(volatile int*)&s.abort;
      if (!ok) break;
      if (n % 64 == 0 || a.wait_ns < kShortLimitNs) {
        if (t0 == 0) t0 = globaltimer_ns();
        if (globaltimer_ns() - t0 > a.wait_ns) {
          *(volatile int*)&s.abort = 1;
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

// ------------------------------------------------------------------------------------------------
// prep: block 0 clears the counters, blocks 1 .. T bring the tokens' rows into the operand's form (unless they are given so), the others
// make the router's logits, of one expert and TT tokens each

constexpr int PREP_THREADS = 256, PREP_TOKENS = 4;  // (four experts to a block as well: no difference at 16 tokens)

template <class F, int TT>
__global__ void __launch_bounds__(PREP_THREADS) prep_kernel(FewArgs a) {
  __shared__ float s_part[PREP_THREADS / 32][TT];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < a.n_counters; i += PREP_THREADS) a.counters[i] = 0;
    return;
  }
  const int row_blocks = a.x_made != nullptr ? a.T : 0;
  if ((int)blockIdx.x <= row_blocks) {
    const int t = blockIdx.x - 1, blocks = a.H / F::KB;
    for (int kb = warp; kb < blocks; kb += PREP_THREADS / 32) {
      const uint16_t* x = a.x + (size_t)t * a.H + kb * F::KB + lane * F::LANE;
      float v[F::LANE];
#pragma unroll
      for (int j = 0; j < F::LANE / 4; ++j) {
        const uint2 w = reinterpret_cast<const uint2*>(x)[j];
        v[4 * j] = bf16_lo(w.x);
        v[4 * j + 1] = bf16_hi(w.x);
        v[4 * j + 2] = bf16_lo(w.y);
        v[4 * j + 3] = bf16_hi(w.y);
      }
      F::write_block(v, a.x_made, a.x_scales_made, t, kb, blocks, blocks);
    }
    return;
  }
  // one expert's logits of TT tokens: its router row is read once, the tokens' rows come from the caches
  const int at = blockIdx.x - 1 - row_blocks, e = at % a.E, t0 = at / a.E * TT;
  float acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.f;
  const int n = a.H / 8;
  const uint4* w = reinterpret_cast<const uint4*>(a.w_router) + (size_t)e * n;
  const uint4* x = reinterpret_cast<const uint4*>(a.x) + (size_t)t0 * n;
#pragma unroll (TT == 1 ? 3 : 1)
  for (int i = threadIdx.x; i < n; i += PREP_THREADS) {
    const uint4 wv = w[i];
    uint4 xv[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) xv[t] = t0 + t < a.T ? x[(size_t)t * n + i] : make_uint4(0, 0, 0, 0);
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint32_t xx[4] = {xv[t].x, xv[t].y, xv[t].z, xv[t].w};
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

MOE_DEV int shared_entries(const FewArgs& a) { return a.Is > 0; }

MOE_DEV void route_rows(const FewArgs& a, Smem& s, Routing& r) {
  const float* logits = a.logits != nullptr ? a.logits : a.logits_ws;
  for (int t = threadIdx.x >> 5; t < a.T; t += WARPS) {
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
// an entry is row p of the activations and of Y.  A shared expert is entry 0, with rows T k .. T k + T - 1.
// r.tokens is zero before, r.held is set.
template <class F>
MOE_DEV void make_entries(const FewArgs& a, Smem& s, Routing& r) {
  constexpr int CHUNKS = MOE_FEW_MAX_EXPERTS / 32, PER = CHUNKS / 8;
  const int slots = a.T * a.k, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  route_rows(a, s, r);
  __syncthreads();
  for (int i = tid; i < slots; i += THREADS) {
    const int e = r.ids[i];
    if (r.held[e]) atomicOr(&r.tokens[e], 1u << (i / a.k));
  }
  __syncthreads();
  const int sh = shared_entries(a);
  uint32_t mine[PER];
  int sums[PER];  // rows and experts << 16: inclusive prefixes over 32 experts
#pragma unroll
  for (int c = 0; c < PER; ++c) {
    const int e = (warp * PER + c) * 32 + lane;
    mine[c] = e < a.E ? r.tokens[e] : 0u;
    sums[c] = __popc(mine[c]) | (mine[c] != 0) << 16;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sums[c], o);
      if (lane >= o) sums[c] += v;
    }
    if (lane == 31 && warp < CHUNKS / PER) r.sums[warp * PER + c] = sums[c];
  }
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < CHUNKS; ++w) {
    if (w < warp * PER) before += r.sums[w];
    all += r.sums[w];
  }
#pragma unroll
  for (int c = 0; c < PER; ++c) {
    const int e = (warp * PER + c) * 32 + lane, m = __popc(mine[c]);
    if (m > 0) {
      const int at = before + sums[c] - (m | 1 << 16), first = at & 0xFFFF;
      r.first[e] = (short)first;
      s.entry[sh + (at >> 16)] = Entry{e - a.first, (short)m, (short)first};
      atomicMax(&s.most, m);
      int q = first;
      for (uint32_t b = mine[c]; b != 0; b &= b - 1, ++q) {
        s.token[q] = (uint8_t)(__ffs(b) - 1);
        s.entry_of[q] = (short)(sh + (at >> 16));
      }
    }
    before += __shfl_sync(0xffffffffu, sums[c], 31);
  }
  if (tid == 0) {
    s.routed = all >> 16;
    s.rows = all & 0xFFFF;
    if (sh) s.entry[0] = Entry{-1, (short)a.T, (short)slots};
  }
  if (sh && tid < a.T) s.token[slots + tid] = (uint8_t)tid;
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

// The units, in the order in which they are drawn: the gate/up units, of the shared expert, then of the routed entries,
// each by rows, then by slices of k; then the down units in the same order.  (Down units that come sooner would stop the
// stream of weights at the activations that they wait for.)
struct Units {
  int sh, shared, gate_up, total, per_gu, per_down;
  MOE_DEV Units(const FewArgs& a, int routed) {
    sh = shared_entries(a);
    per_gu = a.I / 128 * a.slices[0];
    per_down = (a.H + 255) / 256 * a.slices[1];
    shared = a.Is / 128 * a.slices[0];
    gate_up = shared + routed * per_gu;
    total = gate_up + (sh + routed) * per_down;
  }
};

template <class F>
MOE_DEV Unit unit_at(const FewArgs& a, const Smem& s, const Units& us, int u) {
  Unit un;
  const bool down = u >= us.gate_up;
  int v = u;
  un.entry = 0;
  if (down) {
    v -= us.gate_up;
    un.entry = v / us.per_down;
    v -= un.entry * us.per_down;
  } else if (u >= us.shared) {
    v -= us.shared;
    un.entry = v / us.per_gu;
    v -= un.entry * us.per_gu;
    un.entry += us.sh;
  }
  const Entry en = s.entry[un.entry];
  un.expert = en.expert;
  un.m = en.m;
  un.first = en.first;
  un.flags = (down ? DOWN : 0) | (en.expert < 0 ? SHARED : 0);
  const int slices = down ? a.slices[1] : a.slices[0], each = down ? a.slice_blocks[1] : a.slice_blocks[0];
  un.place = v / slices;
  un.slice = v - un.place * slices;
  const int groups = (down ? (en.expert < 0 ? a.Is : a.I) : a.H) / F::KB;
  un.kb0 = min(groups, un.slice * each);
  un.kb1 = min(groups, un.kb0 + each);  // (none: another expert has more slices; its sums are zeros)
  return un;
}

// Draws units, says what they are, and streams their weights.
template <class F>
MOE_DEV void load_weights(const FewArgs& a, const typename F::Maps& maps, Smem& s, uint32_t stages, int u0, int u1) {
  const int lane = lane_id();
  const Units us(a, s.routed);
  int i = 0, n = 0;
  auto load = [&](int drawn) {  // false: there is nothing left, or a wait ran out
    const int u = __shfl_sync(0xffffffffu, drawn, 0), slot = n % DRAWN;
    if (!warp_wait(s.spent[slot], (n / DRAWN & 1) ^ 1, s, a)) return false;
    Unit un = {};
    un.flags = END;
    if (u < us.total) un = unit_at<F>(a, s, us, u);
    if (lane == 0) {
      s.unit[slot] = un;
      mbar_arrive(smem_u32(&s.drawn[slot]));
    }
    ++n;
    if (un.flags & END) return false;
    typename F::Weights weights(a, maps, un);
    for (int kb = un.kb0; kb < un.kb1; ++kb, ++i) {
      const int st = i % NS;
      if (!warp_wait(s.empty[st], (i / NS & 1) ^ 1, s, a)) return false;
      weights.load(kb, stages + st * F::STAGE, smem_u32(&s.full[st]));
    }
    return true;
  };
  // two draws are under way while another's copies are issued
  for (;;) {
    if (!load(u0)) break;
    u0 = draw(a.counters);
    if (!load(u1)) break;
    u1 = draw(a.counters);
  }
  if (lane == 0) s.weights_issued = i;
}

// Loads the activation rows and all scales of the same k blocks, once they are there.
template <class F>
MOE_DEV void load_rows(const FewArgs& a, const typename F::Maps& maps, Smem& s, uint32_t stages) {
  const int lane = lane_id();
  int i = 0, seen = -1;
  for (int n = 0;; ++n) {
    const int slot = n % DRAWN;
    if (!warp_wait(s.drawn[slot], n / DRAWN & 1, s, a)) break;
    const Unit un = s.unit[slot];
    if (un.flags & END) break;
    typename F::Rows rows(a, maps, un);
    bool ok = true;
    if (un.flags & DOWN && un.entry != seen) {
      ok = wait_count(a.ready + un.entry, un.m * ((un.flags & SHARED ? a.Is : a.I) / F::KB), s, a);
      seen = un.entry;
    }
    if (!ok) break;
    rows.start(s, un);
    for (int kb = un.kb0; kb < un.kb1; ++kb, ++i) {
      const int st = i % NS;
      ok = warp_wait(s.empty[st], (i / NS & 1) ^ 1, s, a);
      if (!ok) break;
      rows.load(s, un, kb, stages + st * F::STAGE, s.scales[i % NF], smem_u32(&s.full[st]));
    }
    if (!ok) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.spent[slot]));
  }
  cp_async_commit();
  cp_async_wait<0>();
  if (lane == 0) s.rows_issued = i;
}

// Issues the MMAs of every stage, with an accumulator to each k block.
template <class F>
MOE_DEV void multiply(const FewArgs& a, Smem& s, uint32_t stages) {
  const int nd = F::accumulators(s.most);
  int i = 0, db = 0, turn = 0;
  bool ok = true;
  for (int n = 0; ok; ++n) {
    const int slot = n % DRAWN;
    ok = warp_wait(s.drawn[slot], n / DRAWN & 1, s, a);
    if (!ok) break;
    const int flags = s.unit[slot].flags, blocks = s.unit[slot].kb1 - s.unit[slot].kb0, m = s.unit[slot].m;
    __syncwarp();
    if (flags & END) break;
    if (lane_id() == 0) mbar_arrive(smem_u32(&s.spent[slot]));
    for (int j = 0; j < blocks; ++j, ++i) {
      const int st = i % NS;
      ok = warp_wait(s.full[st], i / NS & 1, s, a) && warp_wait(s.d_empty[db], turn ^ 1, s, a);
      if (!ok) break;
      fence_proxy_async_shared();  // (the rows came through the generic proxy)
      tc_fence_after();
      if (elect_one()) {
        F::multiply(s.tmem, db, stages + st * F::STAGE, m, s.most);
        mma_commit(smem_u32(&s.d_full[db]));
        mma_commit(smem_u32(&s.empty[st]));
      }
      __syncwarp();
      if (++db == nd) {
        db = 0;
        turn ^= 1;
      }
    }
  }
}

// Scales and adds up a unit's accumulators, stores its sums, and publishes them.
template <class F>
MOE_DEV void epilogue(const FewArgs& a, Smem& s) {
  const int lane = lane_id(), warp = threadIdx.x >> 5, q = warp & 3, wr = q * 32 + lane;
  const uint32_t lane_base = s.tmem + ((uint32_t)(q * 32) << 16);
  const int nd = F::accumulators(s.most);
  int i = 0, db = 0, turn = 0;
  for (int n = 0;; ++n) {
    const int slot = n % DRAWN;
    if (!warp_wait(s.drawn[slot], n / DRAWN & 1, s, a)) return;
    const Unit un = s.unit[slot];
    __syncwarp();
    if (un.flags & END) return;
    if (lane == 0) mbar_arrive(smem_u32(&s.spent[slot]));
    uint64_t acc[2][NT / 2];
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) acc[0][j] = acc[1][j] = 0;
    for (int kb = un.kb0; kb < un.kb1; ++kb, ++i) {
      if (!warp_wait(s.d_full[db], turn, s, a)) return;
      tc_fence_after();
      F::add(acc, lane_base, db, s.scales[i % NF], un.m, s.most, smem_u32(&s.d_empty[db]));
      if (++db == nd) {
        db = 0;
        turn ^= 1;
      }
    }
    const float by = F::output_scale(a, un);
    // the slice's sums: [slice][row][2 I] or [slice][row][H]
    const bool down = un.flags & DOWN, is_shared = un.flags & SHARED;
    const int inter = is_shared ? a.Is : a.I, wide = down ? a.H : 2 * inter;
    const int row0 = un.place * (down ? 256 : 128) + wr, row1 = row0 + (down ? 128 : inter);
    float* to = down ? a.Y + un.slice * a.y_slice + (size_t)un.first * wide
                     : is_shared ? a.gu_shared + (size_t)un.slice * a.T * wide
                                 : a.gu + ((size_t)un.slice * a.T * a.k + un.first) * wide;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (j < un.m) {
        float x0, x1;
        unpack_f32x2(acc[0][j / 2], x0, x1);
        to[(size_t)j * wide + row0] = by * (j & 1 ? x1 : x0);
        unpack_f32x2(acc[1][j / 2], x0, x1);
        if (!down || row1 < a.H) to[(size_t)j * wide + row1] = by * (j & 1 ? x1 : x0);
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.stored[slot]));
  }
}

// Publishes the units whose sums are stored.  (A warp of its own: until the stores have arrived in L2 it takes some
// 2 us between the weights' loads, and 7 us where those saturate the memory.)
template <class F>
MOE_DEV void publish(const FewArgs& a, Smem& s) {
  for (int n = 0;; ++n) {
    const int slot = n % DRAWN;
    if (!warp_wait(s.drawn[slot], n / DRAWN & 1, s, a)) return;
    const int flags = s.unit[slot].flags, entry = s.unit[slot].entry, place = s.unit[slot].place;
    if (flags & END) return;
    if (!warp_wait(s.stored[slot], n / DRAWN & 1, s, a)) return;
    __syncwarp();
    if (lane_id() == 0) {
      mbar_arrive(smem_u32(&s.spent[slot]));
      counter_add_release(flags & DOWN ? a.columns_done + place : a.block_done + entry * a.blocks_max + place * 128 / F::KB, 1);
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------------------------------------------
// few: what follows the products

// All units of a block of KB activations of an entry are stored: the whole warp adds up the slices of its row r, makes
// the activations, and brings them into the down products' form.
template <class F>
MOE_DEV void finish_block(const FewArgs& a, Smem& s, int entry, int kb, int r) {
  constexpr int QUADS = F::LANE / 4, AT_ONCE = 4 / QUADS;
  const Entry en = s.entry[entry];
  const bool is_shared = en.expert < 0;
  const int inter = is_shared ? a.Is : a.I, first = is_shared ? 0 : en.first;
  const float limit = is_shared ? a.shared_limit : a.limit;
  const size_t slice = (size_t)(is_shared ? a.T : a.T * a.k) * 2 * inter;
  const float* gu = (is_shared ? a.gu_shared : a.gu) + (size_t)(first + r) * 2 * inter + kb * F::KB + lane_id() * F::LANE;
  float4 gate[QUADS], up[QUADS];
#pragma unroll
  for (int j = 0; j < QUADS; ++j) gate[j] = up[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < a.slices[0]; i0 += AT_ONCE) {
    float4 p[AT_ONCE][QUADS], q[AT_ONCE][QUADS];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (i0 + i < a.slices[0]) {
        const float4* at = reinterpret_cast<const float4*>(gu + (i0 + i) * slice);
#pragma unroll
        for (int j = 0; j < QUADS; ++j) {
          p[i][j] = __ldcg(at + j);
          q[i][j] = __ldcg(at + inter / 4 + j);
        }
      }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (i0 + i < a.slices[0])
#pragma unroll
        for (int j = 0; j < QUADS; ++j) {
          gate[j] = make_float4(gate[j].x + p[i][j].x, gate[j].y + p[i][j].y, gate[j].z + p[i][j].z, gate[j].w + p[i][j].w);
          up[j] = make_float4(up[j].x + q[i][j].x, up[j].y + q[i][j].y, up[j].z + q[i][j].z, up[j].w + q[i][j].w);
        }
  }
  float v[F::LANE];
#pragma unroll
  for (int j = 0; j < QUADS; ++j) {
    v[4 * j] = swiglu_keep_nan<false>(gate[j].x, up[j].x, limit);
    v[4 * j + 1] = swiglu_keep_nan<false>(gate[j].y, up[j].y, limit);
    v[4 * j + 2] = swiglu_keep_nan<false>(gate[j].z, up[j].z, limit);
    v[4 * j + 3] = swiglu_keep_nan<false>(gate[j].w, up[j].w, limit);
  }
  F::write_block(v, is_shared ? a.act_codes_shared : a.act_codes, is_shared ? a.act_scales_shared : a.act_scales,
                 first + r, kb, inter / F::KB, F::scale_pitch(inter / F::KB));
  __syncwarp();
  if (lane_id() == 0) counter_add_release(a.ready + entry, 1);
}

// All units of 32 columns of the result are stored: the whole warp adds up slices and experts of token t, a lane to a
// column, of several slots and slices at once (their loads take a round trip to L2).  The sums of a slot first, in the
// order of its slices, then the slots in theirs.
MOE_DEV void finish_columns(const FewArgs& a, Smem& s, int place, int t) {
  constexpr int SLOTS = 8, SLICES = 2;
  constexpr uint32_t NONE = ~0u;
  const int h = place * 32 + (threadIdx.x & 31);
  float v = 0.f;
  for (int c0 = 0; c0 < a.k; c0 += SLOTS) {
    float sum[SLOTS];
    uint32_t at[SLOTS];  // of the slot's row (at most 528 of them), or NONE
#pragma unroll
    for (int c = 0; c < SLOTS; ++c) {
      const int p = c0 + c < a.k ? s.pos[t * a.k + c0 + c] : -1;
      at[c] = p >= 0 ? (uint32_t)p * a.H + h : NONE;
      sum[c] = 0.f;
    }
    const float* Y = a.Y;
    for (int i0 = 0; i0 < a.slices[1]; i0 += SLICES, Y += SLICES * a.y_slice) {
      float y[SLICES][SLOTS];
#pragma unroll
      for (int i = 0; i < SLICES; ++i)
#pragma unroll
        for (int c = 0; c < SLOTS; ++c)
          y[i][c] = at[c] != NONE && i0 + i < a.slices[1] ? __ldcg(Y + i * a.y_slice + at[c]) : 0.f;
#pragma unroll
      for (int i = 0; i < SLICES; ++i)
#pragma unroll
        for (int c = 0; c < SLOTS; ++c) sum[c] += y[i][c];
    }
#pragma unroll
    for (int c = 0; c < SLOTS; ++c)
      if (at[c] != NONE) v = __fmaf_rn(s.wts[t * a.k + c0 + c], sum[c], v);
  }
  if (a.Is > 0)
    for (int i = 0; i < a.slices[1]; ++i) v += __ldcg(a.Y + (size_t)(a.T * a.k + t) * a.H + h + i * a.y_slice);
  const size_t o = (size_t)t * a.H + h;
  if (a.shared_out != nullptr) v += __bfloat162float(__ushort_as_bfloat16(a.shared_out[o]));
  a.out[o] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Finishes what all its units are stored of: each entry's blocks of activations, row by row, then the columns of the
// result, drawn in this order.  Two warps of a CTA do so from the start, the others when their own work is done.
// (A task of all of an expert's rows takes too long where it has many: 16 tokens at 8 experts, all picked by all, took
// 92 us in FP8 so, and 74 by rows.)
template <class F>
MOE_DEV void finish(const FewArgs& a, Smem& s, int drawn) {
  const int sh = shared_entries(a), entries = s.routed + sh, per_row = a.I / F::KB, places = a.H / 32;
  const int shared_blocks = sh * a.T * (a.Is / F::KB), blocks = shared_blocks + s.rows * per_row;
  const int total = blocks + places * a.T;
  for (;;) {
    const int u = __shfl_sync(0xffffffffu, drawn, 0);
    if (u >= total) return;
    drawn = draw(a.counters + 32);
    if (u >= blocks) {
      const int t = (u - blocks) / places, place = u - blocks - t * places;
      if (!wait_count(a.columns_done + place * 32 / 256, entries * a.slices[1], s, a)) return;
      finish_columns(a, s, place, t);
    } else {
      int v = u, e = 0, m = a.T;
      if (u >= shared_blocks) {
        v -= shared_blocks;
        e = s.entry_of[v / per_row];
        m = s.entry[e].m;
        v -= s.entry[e].first * per_row;
      }
      const int kb = v / m;
      if (!wait_count(a.block_done + e * a.blocks_max + kb, a.slices[0] * F::KB / 128, s, a)) return;
      finish_block<F>(a, s, e, kb, v - kb * m);
    }
  }
}

// After a wait that ran out, whichever, and with all roles ended: waits for the copies and MMAs that are on their way, as
// none may be in a CTA that is gone.  One loader may have ended ahead of the other, or both after others gave up: the
// arrivals that a stage is short of are made here.
template <class F>
MOE_DEV void drain(Smem& s) {
  if (threadIdx.x >> 5 == 1) {  // (the elected lane is the one that has issued the MMAs)
    if (elect_one()) {
      mma_commit(smem_u32(&s.drain));
      mbar_wait_drain(smem_u32(&s.drain), 0);
    }
    __syncwarp();
  } else if (threadIdx.x == 0) {
    const int weights = s.weights_issued, rows = s.rows_issued, end = max(weights, rows);
    for (int j = max(0, end - NS); j < end; ++j) {
      const uint32_t full = smem_u32(&s.full[j % NS]);
      const int missing = (j >= weights ? F::WEIGHT_ARRIVALS : 0) + (j >= rows ? F::FULL_ARRIVALS - F::WEIGHT_ARRIVALS : 0);
      for (int n = 0; n < missing; ++n) mbar_arrive(full);
      mbar_wait_drain(full, j / NS & 1);
    }
  }
}

template <class F>
__global__ void __launch_bounds__(THREADS, PER_SM) few_kernel(const __grid_constant__ FewArgs a,
                                                               const __grid_constant__ typename F::Maps maps) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Smem s;
  const uint32_t stages = (smem_u32(smem) + 1023) / 1024 * 1024;
  Routing& r = *reinterpret_cast<Routing*>(smem + (stages - smem_u32(smem)));
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&s.full[i]), F::FULL_ARRIVALS);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < ND; ++i) {
      mbar_init(smem_u32(&s.d_full[i]), 1);
      mbar_init(smem_u32(&s.d_empty[i]), 4);
    }
    for (int i = 0; i < DRAWN; ++i) {
      mbar_init(smem_u32(&s.drawn[i]), 1);
      mbar_init(smem_u32(&s.spent[i]), 7);  // loader, MMA issuer, epilogue, publisher
      mbar_init(smem_u32(&s.stored[i]), 4);
    }
    mbar_init(smem_u32(&s.drain), 1);
    s.weights_issued = s.rows_issued = 0;
    s.abort = 0;
    s.most = shared_entries(a) ? a.T : 0;  // (from here on raised by atomics alone, of every warp that has picked experts)
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s.tmem), F::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0) F::prefetch(a, maps);
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    r.tokens[e] = 0;
    r.held[e] = F::held(a, e);
  }
  // (A CTA whose tensor memory another kernel's CTA on its SM still has would keep what it has drawn until that one is
  // gone, and all others waiting: it draws once it can work.  The grid before this one hides the barrier.)
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  // (the first draws' answers come while the tokens are routed)
  int u0 = 0, u1 = 0;
  if (warp == 0) {
    u0 = draw(a.counters);
    u1 = draw(a.counters);
  } else if (warp >= 8) {
    u0 = draw(a.counters + 32);
  }
  make_entries<F>(a, s, r);
  fence_proxy_async_shared();  // (the stages' first bytes were the routing's)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s.routed + shared_entries(a) == 0) {  // no expert of this part was picked
    for (int64_t i = blockIdx.x * THREADS + threadIdx.x; i < (int64_t)a.T * a.H; i += (int64_t)gridDim.x * THREADS)
      a.out[i] = a.shared_out != nullptr ? a.shared_out[i] : 0;
  } else if (warp == 0) {
    load_weights<F>(a, maps, s, stages, u0, u1);
  } else if (warp == 1) {
    multiply<F>(a, s, stages);
  } else if (warp < 6) {
    epilogue<F>(a, s);
  } else if (warp == 6) {
    load_rows<F>(a, maps, s, stages);
  } else if (warp == 7) {
    publish<F>(a, s);
  }
  // (the whole warp or none of it)
  if (s.routed + shared_entries(a) > 0 && !__any_sync(0xffffffffu, *(volatile int*)&s.abort))
    finish<F>(a, s, warp >= 8 ? u0 : draw(a.counters + 32));
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (s.abort) drain<F>(s);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(s.tmem, F::TMEM_COLS);
  }
}

template <class F>
int launch(const FewArgs& a, const typename F::Maps& maps, cudaStream_t st) {
  const int nsm = device_sm_count();
  if (nsm <= 0) return MOE_ERR_CUDA;
  constexpr int smem = 1024 + NS * F::STAGE;
  static_assert(PER_SM * (smem + sizeof(Smem) + 1024) <= 228 * 1024 && PER_SM * F::TMEM_COLS <= 512, "CTAs per SM");
  static_assert(NS * F::STAGE >= (int)sizeof(Routing), "the routing has its arrays in the stages");
  using Prep = void (*)(FewArgs);
  const Prep preps[2] = {prep_kernel<F, 1>, prep_kernel<F, PREP_TOKENS>};
  static std::atomic<uint64_t> configured{0};  // a bit per device
  const int dev = current_device_index();
  if (dev < 0) return MOE_ERR_CUDA;
  if (!(configured.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    if (cudaFuncSetAttribute(few_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return MOE_ERR_CUDA;
    // (an SM changes its split of L1 and shared memory only when it is empty: with its own split the prep kernel
    // would have to leave an SM before the other's CTA could be resident there)
    for (Prep p : preps)
      if (cudaFuncSetAttribute(p, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess) return MOE_ERR_CUDA;
    configured.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  }
  const int tokens = a.T == 1 ? 1 : PREP_TOKENS;
  const int blocks = 1 + (a.x_made != nullptr ? a.T : 0) + (a.logits == nullptr ? a.E * ((a.T + tokens - 1) / tokens) : 0);
  const Prep prep = preps[a.T == 1 ? 0 : 1];  // (one token by the other: 46.7 us instead of 45.9)
  const int rc = launch_pdl(prep, dim3(blocks), dim3(PREP_THREADS), 0, st, a);
  if (rc != MOE_OK) return rc;
  return launch_pdl(few_kernel<F>, dim3(nsm * PER_SM), dim3(THREADS), smem, st, a, maps);
}

// The SMs of a whole GB300, whatever the device at hand: the slices of k are the order of the sums and the size of the
// workspace, which is asked for without a device, and neither may change with a part of a GPU.
constexpr int SLICED_FOR_SMS = 152;

// K blocks of a slice over `blocks` of them, of a phase of `units` units a slice: 8 (256 KB to a unit), and half of that,
// or down to `least`, where it would leave the CTAs fewer than two units each (four each: 16 tokens at 24 experts 102 us
// in FP8 instead of 100; one token with at least 2 k blocks in FP8 46 us, with 4 45, in NVFP4 with 1 45, with 2 41).
inline int slice_blocks(int blocks, int64_t units, int least) {
  int want = 8;
  while (want > least && units * ((blocks + want - 1) / want) < 2 * SLICED_FOR_SMS * PER_SM) want /= 2;
  const int slices = (blocks + want - 1) / want;
  return (blocks + slices - 1) / slices;
}

// Workspace: offsets of the buffers; every counter is cleared by each call.
template <class F>
FewLayout layout(int T, int H, int I, int Is, int E, int k) {
  FewLayout l = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += (bytes + 255) / 256 * 256;
    return was;
  };
  const size_t entries = (size_t)std::min(E, T * k) + (Is > 0), slots = (size_t)T * k;
  const int wide = H / F::KB, deep = std::max(I, Is) / F::KB;
  l.slice_blocks[0] = slice_blocks(wide, (int64_t)entries * (I / 128), F::LEAST);
  l.slice_blocks[1] = slice_blocks(deep, (int64_t)entries * ((H + 255) / 256), F::LEAST);
  l.slices[0] = (wide + l.slice_blocks[0] - 1) / l.slice_blocks[0];
  l.slices[1] = (deep + l.slice_blocks[1] - 1) / l.slice_blocks[1];
  l.blocks_max = deep;
  l.n_ready = (int)entries;
  l.n_blocks = (int)(entries * deep);
  l.n_columns = (H + 255) / 256;
  l.n_counters = 64 + l.n_ready + l.n_blocks + l.n_columns;
  l.y_slice = (slots + (Is > 0 ? T : 0)) * H;
  l.counters = take(4 * (size_t)l.n_counters);
  l.logits = take(4 * (size_t)T * E);
  l.x_values = take((size_t)T * wide * F::BLOCK_BYTES);
  l.x_scales = take(4 * (size_t)T * wide);
  l.gu = take(4 * l.slices[0] * slots * 2 * I);
  l.act_values = take(slots * (I / F::KB) * F::BLOCK_BYTES);
  l.act_scales = take(4 * slots * F::scale_pitch(I / F::KB));
  l.gu_shared = take(4 * l.slices[0] * (size_t)T * 2 * Is);
  l.act_values_shared = take((size_t)T * (Is / F::KB) * F::BLOCK_BYTES);
  l.act_scales_shared = take(4 * (size_t)T * F::scale_pitch(Is / F::KB));
  l.Y = take(4 * l.slices[1] * l.y_slice);
  l.total = at;
  return l;
}

// Sets the workspace's pointers.
inline void place(FewArgs& a, const FewLayout& l, void* ws) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  auto floats = [&](size_t at) { return reinterpret_cast<float*>(base + at); };
  a.counters = reinterpret_cast<int*>(base + l.counters);
  a.ready = a.counters + 64;  // (on lines of their own behind the counters that units and tasks are drawn from)
  a.block_done = a.ready + l.n_ready;
  a.columns_done = a.block_done + l.n_blocks;
  a.n_counters = l.n_counters;
  a.blocks_max = l.blocks_max;
  for (int i = 0; i < 2; ++i) {
    a.slices[i] = l.slices[i];
    a.slice_blocks[i] = l.slice_blocks[i];
  }
  a.y_slice = l.y_slice;
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
}

}  // namespace few
}  // namespace moe
