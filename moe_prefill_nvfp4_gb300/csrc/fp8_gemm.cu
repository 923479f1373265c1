// fp8_gemm.cu -- block-scaled FP8 (E4M3) products on the 5th-generation tensor cores, dense and
// grouped by expert:
//
//   C[p, n] = sum_g sa[row(p), g] * sw_e[n / 128, g] * P_g,   P_g = sum_{k in block g} A[row(p), k] W_e[n, k]
//
// A is E4M3 with one FP32 scale per row and 128 columns, W_e E4M3 with one per 128 x 128 block.
// The scales change every 128 k, so a k block is the unit of the accumulation: four
// tcgen05.mma.kind::f8f6f4 (k 32 each) make P_g in tensor memory, the epilogue warps read it and
// add sa * sw * P_g to FP32 registers while the MMAs of the next block run into the other half of
// tensor memory.  Sums stay in FP32 throughout; one rounding makes the BF16 output.
//
// Two kernels:
//   wide  token rows are the MMA's M operand (128 per tile, a TMEM lane and two epilogue threads to a
//         row: its sa is one number), weight rows the N operand (NB blocks of 128, sw uniform over a
//         block).  Persistent CTAs over all experts' tiles (or one tile to a cluster that shares its k
//         blocks, where tiles are few and long).  Bound by shared memory: a k block of a
//         128 x 256 tile is 512 cycles of MMA, and 768 of writing its 48 KB there and reading them
//         back; it takes ~850 (434 ns), 2.9 of the 3.8 PFLOP/s that a library product with one scale
//         to a tensor reaches.  (CTA pairs, whose tiles need 32 KB to an SM, measured slower: with 256
//         columns to an accumulator a k block waits for its release across the pair, 19456 x 1536 x
//         5120 in 123 us against 115; four accumulators of 128 columns take 144.)
//   few   weight rows are the M operand (two blocks of 128 per tile), up to NT token rows the N
//         operand: a tile of the wide kernel would be mostly empty rows.  Bound by the weights' bytes.
//
// Measured on GB300 (GLM sizes: 160 experts, top-8, hidden 5120, intermediate 1536), cold weights, the kernels
// alone (in CUDA graphs of 12 launches, some 20 ms of them):
//   down product      1 token 15.1 us, 64 tokens 182 us (6.6 TB/s), 8192 tokens 577 us (1.8 PFLOP/s)
//   gate/up + SwiGLU  4 tokens 81 us, 64 tokens 352 us (6.9 TB/s), 8192 tokens 1102 us (1.9 PFLOP/s; with
//                     rows that need no gathering 1014)
//   dense             8192 x 1536 x 5120 58 us (2.2 PFLOP/s), 1 x 5120 x 1536 5.8 us
// In a loop of seconds the power limit takes the SM clock from 2.07 to 1.68 GHz and the 8192-token products
// to 607 and 1215 us.
//
// gate/up form: the tile's two blocks are a gate block and the matching up block, and the tile's
// output is a 128-column group of act = silu(min(g, L)) * clamp(u, -L, L), quantised in the
// epilogue (the group's scale needs only this tile), so no intermediate goes to memory.
//
// Operands are staged by TMA in the canonical 128-byte-swizzled K-major layout (one swizzle row is
// one 128-k block).  Out-of-range k, weight rows and tokens are zero-filled by the TMA or hold
// other rows' data that only reaches accumulator rows nobody stores.  Every wait is bounded
// (MOE_DEVERR_TIMEOUT; the CTA then drains its copies and MMAs, frees TMEM and returns).

#include <algorithm>
#include <atomic>

#include "expert_rows.h"
#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace f8 {

constexpr int BK = 128;               // k per stage = one scale block = one 128-byte swizzle row
constexpr int BLK = 128 * BK;         // 128 rows of a stage: 16 KB
constexpr int MAX_E = MOE_FP8_MAX_EXPERTS;

// kind::f8f6f4: D FP32 (bits 4-5 = 1), A and B E4M3 (0), both K-major, N>>3 at 17, M>>4 at 24
__host__ __device__ constexpr uint32_t make_idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// One k block: four k32 MMAs, both descriptors advancing 32 bytes inside the swizzle row; the
// first overwrites D.
MOE_DEV void mma4_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
      " setp.ne.b32 p, 0, 0;\n setp.eq.b32 q, 0, 0;\n"
      " add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
      " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, q;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, q;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc)
      : "memory");
}

MOE_DEV void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Waits for this thread's TMEM loads; naming the registers keeps their uses behind the wait.
template <int N>
MOE_DEV void tmem_wait_ld_regs(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

MOE_DEV void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Two FP32 sums in one 64-bit register pair: acc += {v0, v1} * {f, f}
MOE_DEV uint64_t pack_f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
MOE_DEV void unpack_f32x2(uint64_t d, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
MOE_DEV void fma_f32x2(uint64_t& acc, uint32_t v0, uint32_t v1, uint64_t f) {
  asm("{\n .reg .b64 d;\n mov.b64 d, {%1, %2};\n fma.rn.f32x2 %0, d, %3, %0;\n}" : "+l"(acc) : "r"(v0), "r"(v1), "l"(f));
}

MOE_DEV uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

MOE_DEV uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <uint32_t N>
MOE_DEV void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
MOE_DEV void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

MOE_DEV bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, uint64_t limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity, kSleepHintNs)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit) {
      *abort_flag = 1;
      set_error(err, MOE_DEVERR_TIMEOUT);
      return false;
    }
  }
}

// By a whole warp, every lane polling (a poll by one lane and a shuffle took longer).
MOE_DEV bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, uint64_t limit) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, err, limit));
}

// Orders generic-proxy accesses of shared memory before later asynchronous ones (TMA, MMA).
MOE_DEV void fence_proxy_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Asynchronous 16-byte copy to shared memory, the first `bytes` of it from global memory, zeros after.
MOE_DEV void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
MOE_DEV void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// One of the barrier's expected arrivals, made when this thread's copies so far have landed.
MOE_DEV void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
MOE_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's committed groups of copies are still on their way.
template <int N>
MOE_DEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ... on a barrier that CTAs of the cluster arrive on (acquire at cluster scope)
MOE_DEV bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
  return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort_flag, err));
}

// named_bar_sync that tells every thread whether any of them had pred set.
MOE_DEV bool named_bar_any(uint32_t id, uint32_t nthreads, bool pred) {
  uint32_t any;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(any)
               : "r"(id), "r"(nthreads), "r"(pred ? 1u : 0u)
               : "memory");
  return any != 0;
}

// Token row of sorted row p (checked: an index outside [0, a_rows) reads row 0 and is recorded).
MOE_DEV int source_row(const Fp8GemmArgs& a, int p) {
  if (a.gather == nullptr) return p;
  const int r = __ldg(a.gather + p);
  if ((unsigned)r < (unsigned)a.a_rows) return r;
  set_error(a.err, MOE_DEVERR_BAD_GATHER);
  return 0;
}

// ------------------------------------------------------------------------------------------------
// Tiles.  Expert e (of this call's e_first .. e_first + e_count) owns tiles tbase[e] .. tbase[e+1]):
// ceil(rows / BT) token tiles x NG weight tiles, weight tiles fastest so that CTAs running together
// share token rows and the expert's weights in L2.

// By one warp: the prefix sum of the experts' tile counts, the total in s_tbase[E].  Offsets that are
// not a non-decreasing sequence from 0 to at most R are recorded and make the total -1 (no tile is
// run, no row written).
MOE_DEV void build_tiles(const Fp8GemmArgs& a, const int* s_offs, int* s_tbase, int BT, int NG) {
  const int lane = lane_id();
  const int per = (a.E + 31) / 32;
  const int e0 = min(a.E, lane * per), e1 = min(a.E, e0 + per);
  int sum = 0;
  bool bad = false;
  for (int e = e0; e < e1; ++e) {
    if (!expert_rows_ok(s_offs[e], s_offs[e + 1], a.R))
      bad = true;
    else if ((unsigned)(e - a.e_first) < (unsigned)a.e_count)
      sum += NG * tiles_of_rows(s_offs[e + 1] - s_offs[e], BT);
  }
  if (lane == 0 && s_offs[0] != 0) bad = true;
  bad = __any_sync(0xffffffffu, bad);
  if (bad && lane == 0) set_error(a.err, MOE_DEVERR_BAD_OFFSETS);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int run = incl - sum;
  for (int e = e0; e < e1; ++e) {
    s_tbase[e] = bad ? 0 : run;
    if (!bad && (unsigned)(e - a.e_first) < (unsigned)a.e_count) run += NG * tiles_of_rows(s_offs[e + 1] - s_offs[e], BT);
  }
  if (lane == 31) s_tbase[a.E] = bad ? -1 : incl;
}

struct Tile {
  int e;    // expert within W
  int p0;   // first sorted row
  int cnt;  // token rows
  int ng;   // weight tile
};

MOE_DEV Tile decode_tile(int g, const Fp8GemmArgs& a, const int* s_offs, const int* s_tbase, int BT, int NG) {
  int lo = 0, hi = a.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_tbase[mid] <= g) lo = mid; else hi = mid - 1;
  }
  const int local = g - s_tbase[lo];
  const int tt = local / NG;
  Tile t;
  t.e = lo - a.e_first;
  t.ng = local - tt * NG;
  t.p0 = s_offs[lo] + tt * BT;
  t.cnt = min(BT, s_offs[lo + 1] - t.p0);
  return t;
}

// First weight row of block h of weight tile ng, and the scale row of that block.
template <int NB>
MOE_DEV int block_row(const Fp8GemmArgs& a, int ng, int h) {
  return a.half ? h * a.half + ng * 128 : (ng * NB + h) * 128;
}

// Rows of experts outside W (expert parallelism: other ranks' experts) read as zeros: sorted rows
// [0, offs[e_first]) and [offs[e_first + e_count], offs[E]), a warp to a row; this one is `warp` of
// `warps` of the grid.
MOE_DEV void zero_absent(const Fp8GemmArgs& a, const int* s_offs, int warp, int warps) {
  const int lane = lane_id();
  const int lo = s_offs[a.e_first], hi = s_offs[a.e_first + a.e_count];
  const int rows = lo + (s_offs[a.E] - hi);
  const int esz = a.half ? 1 : a.c_dtype == MOE_DTYPE_BF16 ? 2 : 4;
  const int64_t bytes = (int64_t)(a.half ? a.half : a.N) * esz;
  for (int r = warp; r < rows; r += warps) {
    const int64_t p = r < lo ? r : hi + (r - lo);
    uint8_t* out = a.half ? a.q + p * a.ld_q : static_cast<uint8_t*>(a.C) + p * a.ldc * esz;
    for (int64_t b = lane * 16; b + 16 <= bytes; b += 512) *reinterpret_cast<uint4*>(out + b) = make_uint4(0, 0, 0, 0);
    for (int64_t b = (bytes & ~15ll) + lane; b < bytes; b += 32) out[b] = 0;
    if (a.half) {
      float scale, inv;
      fp8_scale(0, scale, inv);
      for (int g = lane; g < a.half / 128; g += 32) a.s[p * a.s_row + g * a.s_grp] = scale;
    }
  }
}

// 128 bytes of each of the warp's 32 rows into its staging box (w[8 c ..]: chunks of 16 bytes, chunk c of
// row r at c ^ (r % 8), the 128-byte swizzle of the store's tensor map; free of bank conflicts).
MOE_DEV void stage_row(uint32_t box, int lane, const uint32_t (&w)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 128 + ((c ^ (lane & 7)) << 4)),
                 "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                 : "memory");
}

// Stores a staged box at row `row`, column `col` of the output: asynchronously (columns past N are
// clipped, in pieces of 16 bytes), or, where the tile's rows end inside the box or N inside a piece, with
// plain stores of the rows below nrow.
template <typename T>
MOE_DEV void store_box(uint32_t box, const uint8_t* box_ptr, const CUtensorMap* cmap, T* C, int64_t ldc, int64_t row,
                       int col, int nrow, int N) {
  constexpr int PER = 16 / sizeof(T);
  const int lane = lane_id();
  if (col >= N) return;
  if (nrow >= 32 && (col + 8 * PER <= N || N % PER == 0)) {
    if (lane == 0)
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(cmap), "r"(col),
                   "r"((int)row), "r"(box)
                   : "memory");
    return;
  }
  const int c = lane & 7, n = col + c * PER;
  for (int r = lane >> 3; r < nrow; r += 4) {
    const T* src = reinterpret_cast<const T*>(box_ptr + r * 128 + ((c ^ (r & 7)) << 4));
    T* dst = C + (row + r) * ldc + n;
    if (n + PER <= N) {
      *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
    } else {
      for (int j = 0; n + j < N; ++j) dst[j] = src[j];
    }
  }
}

MOE_DEV void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Waits until this thread's bulk stores have read shared memory / are complete.
MOE_DEV void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
MOE_DEV void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ------------------------------------------------------------------------------------------------
// wide kernel

template <int NB_, bool GATHER_, bool GATE_UP_, bool SPLIT_ = false>
struct WideCfg {
  static constexpr int NB = NB_;           // weight blocks of 128 per tile
  static constexpr bool GATE_UP = GATE_UP_;
  static constexpr bool GATHER = GATHER_;  // token rows through gather ids
  static constexpr bool SPLIT = SPLIT_;    // a tile's k blocks shared by a cluster of 2 or 4 CTAs
  static constexpr int BN = NB * 128;
  // warpgroup 0: TMA, MMA, scales; 1 and 2: epilogue; 3: gathering
  static constexpr int THREADS = GATHER ? 512 : 384;
  static constexpr int STAGE = BLK + NB * BLK;
  // The plain form stages its whole BF16 tile (the FP32 tile in two parts) for asynchronous stores and
  // has a stage less for it: stores from the epilogue warps held up the next tile for 1.4 us of the
  // 7.3 us that a tile of K = 1536 took, the fourth stage is worth 1-2%.
  static constexpr int NS = NB == 1 ? 5 : GATE_UP ? 4 : 3;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int EPI_WARP = GATE_UP ? 2048 : NB * 4096;  // 32 rows x 64 bytes; NB boxes of 32 x 128
  static constexpr int OFF_EPI = NS * STAGE;
  static constexpr int OFF_AMAX = OFF_EPI + 8 * EPI_WARP;      // uint32 [2][128]
  static constexpr int NF = 4;              // k blocks whose scales are held
  static constexpr int F_SLOT = 128 + 4;    // sa of the rows, then sw of the blocks
  static constexpr int OFF_F = OFF_AMAX + 2 * 128 * 4;         // float [NF][F_SLOT]
  static constexpr int OFF_OFFS = OFF_F + NF * F_SLOT * 4;
  static constexpr int OFF_TBASE = OFF_OFFS + (MAX_E + 1) * 4;
  static constexpr int OFF_BAR = (OFF_TBASE + (MAX_E + 1) * 4 + 7) & ~7;
  // full[NS] empty[NS] d_full[2] d_empty[2] drain j
  static constexpr int NBAR = 2 * NS + 6;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static constexpr int SMEM = BYTES + 1024;
  // registers: the launch has 384 x 168 or 512 x 128, the warpgroups share the same number
  static constexpr int REG_LAUNCH = GATHER ? 128 : 168;
  static constexpr int REG_LOW = NB == 1 ? REG_LAUNCH - 32 : GATHER ? 56 : 72;
  static constexpr int REG_HIGH = NB == 1 ? REG_LAUNCH + (GATHER ? 32 : 16) : GATHER ? 200 : 216;
  // partial sums for the cluster's other CTAs, 64-bit words [epilogue warp][32][lane], over the drained stages
  static constexpr int PART_WARP = 32 * 32 * 8;
  static_assert(!SPLIT || (NB == 1 && !GATE_UP && 8 * PART_WARP <= NS * STAGE), "partial sums");
  static_assert((THREADS - 256) * REG_LOW + 256 * REG_HIGH <= THREADS * REG_LAUNCH, "register split");
  static_assert(SMEM > 232448 / 2 && SMEM <= 232448, "one CTA per SM (it takes all of TMEM)");
};

// Warp roles: 0 TMA producer, 1 MMA issuer and TMEM owner, 2 the scales of each k block into shared memory
// (asynchronously and blocks ahead, across tiles too: epilogue threads that loaded their own scales waited
// for L2 in every block, 8192 x 1536 x 5120 in 87 us against 60), 4-11 epilogue, 12-15 gathered token rows.
// Epilogue: warp w reads TMEM lanes 32 (w % 4).., its warpgroup g the columns 64 g .. 64 g + 63 of each
// weight block, so that in the gate/up form a thread holds gate columns and their up columns.
template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    wide_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                const __grid_constant__ CUtensorMap cmap, const __grid_constant__ Fp8GemmArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  constexpr int NS = C::NS, NB = C::NB;
  constexpr bool GATHER = C::GATHER;
  int* s_offs = reinterpret_cast<int*>(smem + C::OFF_OFFS);
  int* s_tbase = reinterpret_cast<int*>(smem + C::OFF_TBASE);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (NS + s); };
  auto d_full = [&](int d) { return bar0 + 8u * (2 * NS + d); };
  auto d_empty = [&](int d) { return bar0 + 8u * (2 * NS + 2 + d); };
  const uint32_t drain_bar = bar0 + 8u * (2 * NS + 4), j_bar = drain_bar + 8;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  float* s_f = reinterpret_cast<float*>(smem + C::OFF_F);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t limit = args.wait_ns;
  int* err = args.err;
  // tiles first, first + step, ...; with SPLIT one tile to a cluster of S CTAs
  const int S = C::SPLIT ? (int)cluster_nctarank() : 1, rank = C::SPLIT ? (int)cluster_ctarank() : 0;
  const int first = C::SPLIT ? (int)cluster_id_x() : (int)blockIdx.x;
  const int step = C::SPLIT ? (int)cluster_count_x() : (int)gridDim.x;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), GATHER ? 1 + 128 : 1);  // TMA; every gathering thread
      mbar_init(empty(s), 1);
    }
    for (int d = 0; d < 2; ++d) {
      mbar_init(d_full(d), 2);   // MMA commit, scales
      mbar_init(d_empty(d), 8);  // the epilogue warps
    }
    mbar_init(drain_bar, 1);
    if (C::SPLIT) mbar_init(j_bar, S);  // the CTAs whose partial sums are written
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  if (C::SPLIT) cluster_sync_all();  // the barriers exist before other CTAs arrive on them
  griddep_wait();
  griddep_launch_dependents();
  const int NG = C::GATE_UP ? args.half / 128 : (args.N + C::BN - 1) / C::BN;
  if (args.offsets == nullptr) {  // dense: one group of R rows
    if (tid == 0) {
      s_offs[0] = 0;
      s_offs[1] = args.R;
    }
  } else {
    for (int i = tid; i <= args.E; i += C::THREADS) s_offs[i] = args.offsets[i];
  }
  __syncthreads();
  if (warp == 0) build_tiles(args, s_offs, s_tbase, 128, NG);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  const int KB = (args.K + BK - 1) / BK;
  const int total = s_tbase[args.E];
  // this CTA's k blocks
  const int kb0 = C::SPLIT ? KB * rank / S : 0, kb1 = C::SPLIT ? KB * (rank + 1) / S : KB;

  if (warp < 4) {
    reg_dec<C::REG_LOW>();
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      if (lane == 0) {
        prefetch_tmap(&amap);
        prefetch_tmap(&wmap);
        int i = 0;
        bool ok = true;
        for (int g = first; ok && g < total; g += step) {
          const Tile t = decode_tile(g, args, s_offs, s_tbase, 128, NG);
          for (int kb = kb0; kb < kb1; ++kb, ++i) {
            const int s = i % NS;
            if (!wait_bounded(empty(s), ((i / NS) & 1) ^ 1, s_abort, err, limit)) {
              ok = false;
              break;
            }
            const uint32_t st = sbase + s * C::STAGE;
            mbar_arrive_expect_tx(full(s), (GATHER ? 0 : BLK) + NB * BLK);
            if (!GATHER) tma_load_2d(st, &amap, kb * BK, t.p0, full(s));
#pragma unroll
            for (int h = 0; h < NB; ++h)
              tma_load_3d(st + BLK + h * BLK, &wmap, kb * BK, block_row<NB>(args, t.ng, h), t.e, full(s));
          }
        }
        // every copy issued lands before the CTA leaves (a stage that misses other arrivals, of gathering
        // threads that gave up too, is waited for until the limit, by which its copies have landed)
        if (!ok)
          for (int j = max(0, i - NS); j < i; ++j)
            if (!mbar_wait_drain(full(j % NS), (j / NS) & 1)) break;
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc = make_idesc_e4m3(128, C::BN);
      int i = 0;
      bool ok = true;
      for (int g = first; ok && g < total; g += step) {
        for (int kb = kb0; kb < kb1; ++kb, ++i) {
          const int s = i % NS, db = i & 1;
          // (the operands are usually there first: the accumulator's release is what an MMA waits for)
          if (!warp_wait(full(s), (i / NS) & 1, s_abort, err, limit)) {
            ok = false;
            break;
          }
          if (GATHER) fence_proxy_async_shared();  // the gathered rows came through the generic proxy
          const uint32_t st = sbase + s * C::STAGE;
          const uint64_t a_desc = make_sdesc_sw128(st), b_desc = make_sdesc_sw128(st + BLK);
          if (!warp_wait(d_empty(db), ((i >> 1) & 1) ^ 1, s_abort, err, limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            mma4_e4m3_ss(tmem_base + (uint32_t)(db * C::BN), a_desc, b_desc, idesc);
            mma_commit(d_full(db));
            mma_commit(empty(s));
          }
          __syncwarp();
        }
      }
      if (!ok) {  // every issued MMA completes before TMEM is freed
        if (elect_one()) {
          mma_commit(drain_bar);
          mbar_wait_drain(drain_bar, 0);
        }
        __syncwarp();
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------------- scales of every k block
      // Block i's copies are issued two blocks ahead, into the slot that block i - 4 left; once the
      // accumulator buffer of block i is free its arrival joins the MMA's commit.
      const float* sa[4];
      const float* sw = nullptr;
      int g = first, kb = kb0, n = 0;  // the next block to copy
      auto copy_next = [&]() {
        if (g < total) {
          if (kb == kb0) {
            const Tile t = decode_tile(g, args, s_offs, s_tbase, 128, NG);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              sa[j] = args.sa + (int64_t)source_row(args, t.p0 + min(32 * j + lane, t.cnt - 1)) * args.sa_row + kb0 * args.sa_grp;
            // lane h < NB: block h's (past N: any scale, the block's columns are not stored)
            const int blk = min(block_row<NB>(args, t.ng, min(lane, NB - 1)) >> 7, args.nblk - 1);
            sw = args.sw + ((int64_t)t.e * args.nblk + blk) * KB;
          }
          const uint32_t dst = sbase + C::OFF_F + (uint32_t)((n % C::NF) * C::F_SLOT + lane) * 4u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            cp_async4(dst + 128u * j, sa[j]);
            sa[j] += args.sa_grp;
          }
          if (lane < NB) cp_async4(dst + 512u, sw + kb);
          if (++kb == kb1) {
            kb = kb0;
            g += step;
          }
          ++n;
        }
        cp_async_commit();  // (an empty group past the last block)
      };
      copy_next();
      copy_next();
      for (int i = 0; i < n; ++i) {
        if (!warp_wait(d_empty(i & 1), ((i >> 1) & 1) ^ 1, s_abort, err, limit)) break;
        cp_async_wait<1>();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_full(i & 1));
        copy_next();
      }
      cp_async_wait<0>();
    }
  } else if (GATHER && warp >= 12) {
    // ------------------------------------------------------------------ gathered token rows
    // 16-byte cp.async into the swizzled layout (chunk c of row r at c ^ (r % 8)): 8 lanes to a row of
    // the k block, 4 rows to an instruction, every fourth group of 4 rows to a warp (gate/up of 2048 tokens at
    // 40 experts 286 us; rows gathered by TMA gather4 689, rows that need no gathering 260).  Sixteens of rows
    // past the tile's are left as they are (their accumulator rows are not stored), single rows repeat its last.
    reg_dec<C::REG_LOW>();
    const int r0 = (warp - 12) * 4 + (lane >> 3);  // rows r0 + 16 j: the same chunk place in all of them
    const int chunk = lane & 7;
    const uint32_t dst = sbase + (uint32_t)(r0 * BK + ((chunk ^ (r0 & 7)) << 4));
    int i = 0;
    bool ok = true;
    for (int g = first; ok && g < total; g += step) {
      const Tile t = decode_tile(g, args, s_offs, s_tbase, 128, NG);
      const uint8_t* src[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        src[j] = args.A + source_row(args, t.p0 + min(r0 + 16 * j, t.cnt - 1)) * args.lda + kb0 * BK + chunk * 16;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int s = i % NS;
        if (!warp_wait(empty(s), ((i / NS) & 1) ^ 1, s_abort, err, limit)) {
          ok = false;
          break;
        }
        const int left = args.K - kb * BK - chunk * 16;
        if (left >= 16) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (16 * j < t.cnt) cp_async16(dst + s * C::STAGE + j * 16 * BK, src[j], 16);
        } else {  // past K: zeros (an address inside the row, of which nothing or the rest is read)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (16 * j < t.cnt)
              cp_async16(dst + s * C::STAGE + j * 16 * BK, left > 0 ? src[j] : args.A, (uint32_t)max(left, 0));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) src[j] += BK;
        cp_async_arrive(full(s));
      }
    }
    cp_async_wait<0>();
  } else {
    // ------------------------------------------------------------------ epilogue
    reg_inc<C::REG_HIGH>();
    const int wg = (warp - 4) >> 2;
    const int q = warp & 3;
    const uint32_t stg = sbase + C::OFF_EPI + (warp - 4) * C::EPI_WARP;
    uint32_t* s_amax = reinterpret_cast<uint32_t*>(smem + C::OFF_AMAX);
    const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(wg * 64);
    const int row = q * 32 + lane;  // of the tile
    if (total >= 0) zero_absent(args, s_offs, (int)blockIdx.x * 8 + warp - 4, (int)gridDim.x * 8);
    int i = 0;
    bool ok = true;
    for (int g = first; ok && g < total; g += step) {
      const Tile t = decode_tile(g, args, s_offs, s_tbase, 128, NG);
      uint64_t acc[NB][32];
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[h][j] = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int db = i & 1;
        if (!warp_wait(d_full(db), (i >> 1) & 1, s_abort, err, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t base = lane_base + (uint32_t)(db * C::BN);
        // 16 columns at a time through three register buffers (column j of this warp's 64 NB is column
        // j % 64 of block j / 64); the accumulator is given back once its last columns are in registers
        constexpr int NV = 3;
        uint32_t v[NV][16];
        auto load = [&](int c) {
          tmem_ld_32x32b_x16(base + (uint32_t)((c >> 2) * 128 + (c & 3) * 16), v[c % NV]);
        };
#pragma unroll
        for (int c = 0; c < NV; ++c) load(c);
        uint64_t f[NB];
#pragma unroll
        for (int h = 0; h < NB; ++h) {
          const float* slot = s_f + (i % C::NF) * C::F_SLOT;
          const float x = slot[row] * slot[128 + h];
          f[h] = pack_f32x2(x, x);
        }
#pragma unroll
        for (int c = 0; c < 4 * NB; c += NV) {
#pragma unroll
          for (int d = 0; d < NV; ++d) tmem_wait_ld_regs(v[d]);
          if (c + NV >= 4 * NB) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(d_empty(db));
          }
#pragma unroll
          for (int d = c; d < c + NV && d < 4 * NB; ++d) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              fma_f32x2(acc[d >> 2][(d & 3) * 8 + j], v[d % NV][2 * j], v[d % NV][2 * j + 1], f[d >> 2]);
            if (d + NV < 4 * NB) load(d + NV);
          }
        }
      }
      // (the gate/up form's warps exchange maxima below: all of them leave the loop at the same tile)
      if (C::GATE_UP || C::SPLIT ? named_bar_any(1, 256, !ok) : !ok) {
        ok = false;
        break;
      }
      if constexpr (C::GATE_UP) {
        const bool live = row < t.cnt;
        // gate (block 0) and up (block 1) columns 64 wg .. of the act group
        float high = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float g0, g1, u0, u1;
          unpack_f32x2(acc[0][j], g0, g1);
          unpack_f32x2(acc[NB - 1][j], u0, u1);
          g0 = swiglu_keep_nan<true>(g0, u0, args.limit);
          g1 = swiglu_keep_nan<true>(g1, u1, args.limit);
          high = max_nan(high, max_nan(fabsf(g0), fabsf(g1)));
          acc[0][j] = pack_f32x2(g0, g1);
        }
        uint32_t m = __float_as_uint(high);
        s_amax[wg * 128 + row] = m;
        named_bar_sync(1, 256);
        m = max(m, s_amax[(wg ^ 1) * 128 + row]);  // (the next tile's write comes after its first barrier)
        float scale, inv;
        fp8_scale(m, scale, inv);
        const uint64_t inv2 = pack_f32x2(inv, inv);
        // This row's 64 codes: a warp's 32 rows leave together through its staging box (16-byte chunk c of
        // row r at c ^ ((r >> 1) % 4), the 64-byte swizzle), rows where the tile ends each by itself.
        const int nrow = t.cnt - q * 32, col = t.ng * 128 + wg * 64;
        if (nrow >= 32) {
          if (lane == 0) bulk_wait_read();  // the last box has left
          __syncwarp();
        }
        uint8_t* dst = args.q + (int64_t)(t.p0 + row) * args.ld_q + col;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float a0, a1, a2, a3;
            unpack_f32x2(mul_f32x2(acc[0][c * 8 + 2 * j], inv2), a0, a1);
            unpack_f32x2(mul_f32x2(acc[0][c * 8 + 2 * j + 1], inv2), a2, a3);
            w[j] = pack_e4m3x4(a0, a1, a2, a3);
          }
          if (nrow >= 32)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
          else if (live)
            *reinterpret_cast<uint4*>(dst + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (nrow >= 32) {
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(&cmap),
                         "r"(col), "r"(t.p0 + q * 32), "r"(stg)
                         : "memory");
            bulk_commit();
          }
        }
        if (live && wg == 0) args.s[(int64_t)(t.p0 + row) * args.s_row + t.ng * args.s_grp] = scale;
      } else if constexpr (C::SPLIT) {
        // Of each thread's 64 columns, sixteens 4 rank / S .. are this CTA's to sum and store: the others'
        // go to shared memory (the stages are drained: every accumulator has been read).
        const uint32_t part = sbase + (uint32_t)((warp - 4) * C::PART_WARP + lane * 8);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (b * S / 4 != rank)
#pragma unroll
            for (int j = 8 * b; j < 8 * b + 8; ++j)
              asm volatile("st.shared.b64 [%0], %1;" ::"r"(part + (uint32_t)(j * 256)), "l"(acc[0][j]) : "memory");
        named_bar_sync(1, 256);
        if (tid == 128)
          for (int c = 0; c < S; ++c) mbar_arrive_remote(j_bar, (uint32_t)c);
        if (!warp_wait_cluster(j_bar, 0, s_abort, err)) break;
        const bool live = row < t.cnt;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (b * S / 4 != rank) continue;
          for (int c = 0; c < S; ++c) {  // in the order of the ranks, this CTA's own first
            if (c == rank) continue;
            uint32_t at;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(part), "r"(c));
            uint64_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v[j]) : "r"(at + (uint32_t)((8 * b + j) * 256)));
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[0][8 * b + j] = add_f32x2(acc[0][8 * b + j], v[j]);
          }
          const int col = block_row<NB>(args, t.ng, 0) + wg * 64 + 16 * b;
          float o[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) unpack_f32x2(acc[0][8 * b + j], o[2 * j], o[2 * j + 1]);
          const int64_t at = (int64_t)(t.p0 + row) * args.ldc + col;
          if (!live) {
          } else if (col + 16 > args.N) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (col + j < args.N) {
                if (args.c_dtype == MOE_DTYPE_BF16)
                  static_cast<__nv_bfloat16*>(args.C)[at + j] = __float2bfloat16_rn(o[j]);
                else
                  static_cast<float*>(args.C)[at + j] = o[j];
              }
          } else if (args.c_dtype == MOE_DTYPE_BF16) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.C) + at);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              dst[j] = make_uint4(pack_bf16x2(o[8 * j], o[8 * j + 1]), pack_bf16x2(o[8 * j + 2], o[8 * j + 3]),
                                  pack_bf16x2(o[8 * j + 4], o[8 * j + 5]), pack_bf16x2(o[8 * j + 6], o[8 * j + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(args.C) + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
      } else {
        const int nrow = min(32, t.cnt - q * 32);
        const int64_t row0 = t.p0 + q * 32;
        const uint8_t* stg_ptr = smem + (stg - sbase);
        uint32_t w[32];
        if (args.c_dtype == MOE_DTYPE_BF16) {
          if (lane == 0) bulk_wait_read();  // the last tile's boxes have left
          __syncwarp();
#pragma unroll
          for (int h = 0; h < NB; ++h) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              float a0, a1;
              unpack_f32x2(acc[h][j], a0, a1);
              w[j] = pack_bf16x2(a0, a1);
            }
            stage_row(stg + h * 4096, lane, w);
          }
          fence_proxy_async_shared();
          __syncwarp();
#pragma unroll
          for (int h = 0; h < NB; ++h)
            store_box(stg + h * 4096, stg_ptr + h * 4096, &cmap, static_cast<uint16_t*>(args.C), args.ldc, row0,
                      block_row<NB>(args, t.ng, h) + wg * 64, nrow, args.N);
          if (lane == 0) bulk_commit();
          __syncwarp();
        } else {
          // a box holds 32 columns: NB boxes at a time
#pragma unroll
          for (int u = 0; u < 2 * NB; ++u) {  // columns 32 (u % 2).. of block u / 2
            if (u % NB == 0) {
              if (lane == 0) bulk_wait_read();
              __syncwarp();
            }
            const uint32_t box = (uint32_t)(u % NB) * 4096;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float a0, a1;
              unpack_f32x2(acc[u >> 1][(u & 1) * 16 + j], a0, a1);
              w[2 * j] = __float_as_uint(a0);
              w[2 * j + 1] = __float_as_uint(a1);
            }
            stage_row(stg + box, lane, w);
            fence_proxy_async_shared();
            __syncwarp();
            store_box(stg + box, stg_ptr + box, &cmap, static_cast<float*>(args.C), args.ldc, row0,
                      block_row<NB>(args, t.ng, u >> 1) + wg * 64 + (u & 1) * 32, nrow, args.N);
            if (lane == 0) bulk_commit();
            __syncwarp();
          }
        }
      }
    }
    if (!C::SPLIT && lane == 0) bulk_wait();
  }

  tc_fence_before();
  if (C::SPLIT) {
    __syncwarp();
    cluster_sync_all();  // the other CTAs have read this one's sums
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------------------------
// few-row kernel
//
// Bound by the weights it streams.  Persistent, with loads under way across tiles: CTAs of one tile each
// spent ~4 us on their start and end (64 tokens' down product 195 us, persistent 178).  One SM draws 77 GB/s
// from DRAM at most (44.7 is its share when all of them do), so it pays to have every tile's CTA resident at
// once: two CTAs to an SM where their stages fit (192 tiles: 41 us; one CTA with twice the stages 49), k
// split over a cluster where tiles are few.

template <int NT_, int NS_, int PER_SM_>
struct FewCfg {
  static constexpr int NT = NT_;            // token rows per tile
  static constexpr int NS = NS_;
  static constexpr int PER_SM = PER_SM_;    // CTAs per SM
  static constexpr int THREADS = 224;
  static constexpr int STAGE = 2 * BLK + NT * BK;
  // accumulators: a k block of a tile is little work for the MMA and the epilogue, most of its way through
  // both is latency, which eight on their way hide (3% less time than with two)
  static constexpr int ND = 8;
  static constexpr int TMEM_COLS = ND * 2 * NT;
  static constexpr int PART = NT * 256 * 4;  // a tile's partial sums [NT][256] of a cluster, over the drained stages
  static constexpr int AHEAD = 4;           // k blocks that the copies of scales run ahead
  static constexpr int NF = 16;             // k blocks whose scales are held, at least ND + AHEAD
  static constexpr int F_SLOT = NT + 4;     // sa of the rows, then sw of the two blocks
  static constexpr int OFF_F = NS * STAGE;                   // float [NF][F_SLOT]
  static constexpr int OFF_AMAX = OFF_F + NF * F_SLOT * 4;   // uint32 [2][NT][4]
  static constexpr int OFF_OFFS = OFF_AMAX + 2 * NT * 4 * 4;
  static constexpr int OFF_TBASE = OFF_OFFS + (MAX_E + 1) * 4;
  static constexpr int OFF_BAR = (OFF_TBASE + (MAX_E + 1) * 4 + 7) & ~7;
  static constexpr int NBAR = 2 * NS + 2 * ND + 1;  // full[NS] empty[NS] d_full[ND] d_empty[ND] drain
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static constexpr int SMEM = BYTES + 1024;
  static_assert(NF >= ND + AHEAD && TMEM_COLS <= 512 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "accumulators");
  static_assert(NT % 16 == 0 && NT <= 32 && STAGE % 1024 == 0 && F_SLOT % 4 == 0 && PART <= NS * STAGE, "tile");
  static_assert(PER_SM * (SMEM + 1024) <= 228 * 1024 && PER_SM * TMEM_COLS <= 512, "CTAs per SM");
};

// Warp roles: 0 TMA producer, 1 MMA issuer and TMEM owner, 2-5 epilogue (TMEM lanes 32 (w % 4)..), 6 the
// scales of each k block, as in the wide kernel.
// CTAs that are a cluster of their own take tiles g, g + CTAs, ...  A cluster of S > 1 CTAs has one tile:
// CTA `rank` takes its k blocks KB rank / S .. KB (rank + 1) / S, and the partial sums meet in shared memory.
template <class C, bool GATHER>
__global__ void __launch_bounds__(C::THREADS, C::PER_SM)
    few_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
               const __grid_constant__ Fp8GemmArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  constexpr int NS = C::NS, NT = C::NT, ND = C::ND;
  int* s_offs = reinterpret_cast<int*>(smem + C::OFF_OFFS);
  int* s_tbase = reinterpret_cast<int*>(smem + C::OFF_TBASE);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (NS + s); };
  auto d_full = [&](int d) { return bar0 + 8u * (2 * NS + d); };
  auto d_empty = [&](int d) { return bar0 + 8u * (2 * NS + ND + d); };
  const uint32_t drain_bar = bar0 + 8u * (2 * NS + 2 * ND);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t limit = args.wait_ns;
  int* err = args.err;
  const int S = (int)cluster_nctarank(), rank = (int)cluster_ctarank();

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int d = 0; d < ND; ++d) {
      mbar_init(d_full(d), 2);   // MMA commit, scales
      mbar_init(d_empty(d), 4);  // the epilogue warps
    }
    mbar_init(drain_bar, 1);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&amap);
    prefetch_tmap(&wmap);
  }
  griddep_wait();
  griddep_launch_dependents();
  const int NG = args.half ? args.half / 128 : (args.N + 255) / 256;
  if (args.offsets == nullptr) {
    if (tid == 0) {
      s_offs[0] = 0;
      s_offs[1] = args.R;
    }
  } else {
    for (int i = tid; i <= args.E; i += C::THREADS) s_offs[i] = args.offsets[i];
  }
  __syncthreads();
  if (warp == 0) build_tiles(args, s_offs, s_tbase, NT, NG);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  const int KB = (args.K + BK - 1) / BK;
  const int total = s_tbase[args.E];
  const int first = (int)cluster_id_x(), step = (int)cluster_count_x();
  const int kb0 = (int)((int64_t)KB * rank / S), kb1 = (int)((int64_t)KB * (rank + 1) / S);
  float* part = reinterpret_cast<float*>(smem);

  // Output of token n of tile t from this thread's sums v0 (block 0) and v1 (block 1); the gate/up form
  // returns the activation, its token's largest among the warp's in s_amax, and is finished by quantise()
  // once the four epilogue warps have met.
  const int q = warp & 3;
  const int wr = q * 32 + lane;  // weight row of each block
  uint32_t* s_amax = reinterpret_cast<uint32_t*>(smem + C::OFF_AMAX);
  auto store = [&](const Tile& t, int n, float v0, float v1, uint32_t* amax) {
    const int64_t p = t.p0 + n;
    if (args.half) {
      const float act = swiglu_keep_nan<false>(v0, v1, args.limit);
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(act) & 0x7FFFFFFFu);
      if (lane == 0) amax[n * 4 + q] = m;
      return act;
    }
    const int n0 = block_row<2>(args, t.ng, 0) + wr, n1 = n0 + 128;
    if (args.c_dtype == MOE_DTYPE_BF16) {
      __nv_bfloat16* c = static_cast<__nv_bfloat16*>(args.C) + p * args.ldc;
      if (n0 < args.N) c[n0] = __float2bfloat16_rn(v0);
      if (n1 < args.N) c[n1] = __float2bfloat16_rn(v1);
    } else {
      float* c = static_cast<float*>(args.C) + p * args.ldc;
      if (n0 < args.N) c[n0] = v0;
      if (n1 < args.N) c[n1] = v1;
    }
    return 0.f;
  };
  auto quantise = [&](const Tile& t, int n, float act, const uint32_t* amax) {
    const uint4 m4 = *reinterpret_cast<const uint4*>(amax + n * 4);
    float scale, inv;
    fp8_scale(max(max(m4.x, m4.y), max(m4.z, m4.w)), scale, inv);
    const int64_t p = t.p0 + n;
    args.q[p * args.ld_q + t.ng * 128 + wr] = (uint8_t)pack_e4m3x4(act * inv, 0.f, 0.f, 0.f);
    if (wr == 0) args.s[p * args.s_row + t.ng * args.s_grp] = scale;
  };

  bool ok = true;
  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (whole warp)
    int i = 0;
    for (int g = first; ok && g < total; g += step) {
      const Tile t = decode_tile(g, args, s_offs, s_tbase, NT, NG);
      int r[4] = {0, 0, 0, 0};
      const int nrow4 = (t.cnt + 3) >> 2;
      if (GATHER && lane < nrow4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = source_row(args, t.p0 + min(4 * lane + j, t.cnt - 1));
      }
      const uint32_t bytes = 2 * BLK + (GATHER ? nrow4 * 4 : NT) * BK;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int s = i % NS;
        if (!warp_wait(empty(s), ((i / NS) & 1) ^ 1, s_abort, err, limit)) {
          ok = false;
          break;
        }
        const uint32_t st = sbase + s * C::STAGE;
        if (lane == 0) {
          mbar_arrive_expect_tx(full(s), bytes);
          tma_load_3d(st, &wmap, kb * BK, block_row<2>(args, t.ng, 0), t.e, full(s));
          tma_load_3d(st + BLK, &wmap, kb * BK, block_row<2>(args, t.ng, 1), t.e, full(s));
          if (!GATHER) tma_load_2d(st + 2 * BLK, &amap, kb * BK, t.p0, full(s));
        }
        if (GATHER) {
          __syncwarp();
          if (lane < nrow4) tma_gather4(st + 2 * BLK + lane * 4 * BK, &amap, kb * BK, r[0], r[1], r[2], r[3], full(s));
        }
      }
    }
    if (!ok && lane == 0)
      for (int j = max(0, i - NS); j < i; ++j) mbar_wait_drain(full(j % NS), (j / NS) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = make_idesc_e4m3(128, NT);
    int i = 0;
    for (int g = first; ok && g < total; g += step) {
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int s = i % NS, db = i % ND;
        if (!warp_wait(full(s), (i / NS) & 1, s_abort, err, limit) ||
            !warp_wait(d_empty(db), ((i / ND) & 1) ^ 1, s_abort, err, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t st = sbase + s * C::STAGE;
        if (elect_one()) {
          const uint64_t tok = make_sdesc_sw128(st + 2 * BLK);
          mma4_e4m3_ss(tmem_base + (uint32_t)(db * 2 * NT), make_sdesc_sw128(st), tok, idesc);
          mma4_e4m3_ss(tmem_base + (uint32_t)(db * 2 * NT + NT), make_sdesc_sw128(st + BLK), tok, idesc);
          mma_commit(d_full(db));
          mma_commit(empty(s));
        }
        __syncwarp();
      }
    }
    if (!ok) {
      if (elect_one()) {
        mma_commit(drain_bar);
        mbar_wait_drain(drain_bar, 0);
      }
      __syncwarp();
    }
  } else if (warp == 6) {
    // ------------------------------------------------------------------ scales of every k block
    const float* sa = nullptr;
    const float* sw = nullptr;
    int g = first, kb = kb0, n = 0;
    auto copy_next = [&]() {
      if (g < total) {
        if (kb == kb0) {
          const Tile t = decode_tile(g, args, s_offs, s_tbase, NT, NG);
          sa = args.sa + (int64_t)source_row(args, t.p0 + min(lane, t.cnt - 1)) * args.sa_row + kb0 * args.sa_grp;
          const int blk = min(block_row<2>(args, t.ng, lane & 1) >> 7, args.nblk - 1);
          sw = args.sw + ((int64_t)t.e * args.nblk + blk) * KB;
        }
        const uint32_t dst = sbase + C::OFF_F + (uint32_t)((n % C::NF) * C::F_SLOT + lane) * 4u;
        if (lane < NT) cp_async4(dst, sa);
        sa += args.sa_grp;
        if (lane < 2) cp_async4(dst + NT * 4u, sw + kb);
        if (++kb == kb1) {
          kb = kb0;
          g += step;
        }
        ++n;
      }
      cp_async_commit();  // (an empty group past the last block)
    };
    for (int j = 0; j < C::AHEAD; ++j) copy_next();
    for (int i = 0; i < n; ++i) {
      if (!warp_wait(d_empty(i % ND), ((i / ND) & 1) ^ 1, s_abort, err, limit)) break;
      cp_async_wait<C::AHEAD - 1>();
      __syncwarp();
      if (lane == 0) mbar_arrive(d_full(i % ND));
      copy_next();
    }
    cp_async_wait<0>();
  } else {
    // ------------------------------------------------------------------ epilogue
    const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16);
    const float* s_f = reinterpret_cast<const float*>(smem + C::OFF_F);
    int i = 0, tile = 0;
    for (int g = first; ok && g < total; g += step, ++tile) {
      uint64_t acc[2][NT / 2];
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) acc[0][j] = acc[1][j] = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int db = i % ND;
        if (!warp_wait(d_full(db), (i / ND) & 1, s_abort, err, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[2 * NT / 16][16];
#pragma unroll
        for (int c = 0; c < 2 * NT / 16; ++c)
          tmem_ld_32x32b_x16(lane_base + (uint32_t)(db * 2 * NT + c * 16), v[c]);
        const float* slot = s_f + (i % C::NF) * C::F_SLOT;
        uint64_t sa[NT / 2];  // of tokens 2 j and 2 j + 1
#pragma unroll
        for (int j = 0; j < NT / 4; ++j) {
          const ulonglong2 u = reinterpret_cast<const ulonglong2*>(slot)[j];
          sa[2 * j] = u.x;
          sa[2 * j + 1] = u.y;
        }
        const uint64_t sw[2] = {pack_f32x2(slot[NT], slot[NT]), pack_f32x2(slot[NT + 1], slot[NT + 1])};
#pragma unroll
        for (int c = 0; c < 2 * NT / 16; ++c) tmem_wait_ld_regs(v[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty(db));
#pragma unroll
        for (int c = 0; c < 2 * NT / 16; ++c) {  // 16 columns: tokens 16 (c % (NT / 16)).. of block c / (NT / 16)
          constexpr int PER = NT / 16;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            fma_f32x2(acc[c / PER][(c % PER) * 8 + j], v[c][2 * j], v[c][2 * j + 1],
                      mul_f32x2(sa[(c % PER) * 8 + j], sw[c / PER]));
        }
      }
      // (all four warps leave the loop at the same tile)
      if (named_bar_any(1, 128, !ok)) {
        ok = false;
        break;
      }
      if (S > 1) {
        // every k block has been accumulated, so the stages are drained
#pragma unroll
        for (int n = 0; n < NT / 2; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float a0, a1;
            unpack_f32x2(acc[h][n], a0, a1);
            part[(2 * n) * 256 + h * 128 + wr] = a0;
            part[(2 * n + 1) * 256 + h * 128 + wr] = a1;
          }
      } else {
        const Tile t = decode_tile(g, args, s_offs, s_tbase, NT, NG);
        uint32_t* amax = s_amax + (tile & 1) * NT * 4;
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          if (n >= t.cnt) break;
          float g0, g1, u0, u1;
          unpack_f32x2(acc[0][n / 2], g0, g1);
          unpack_f32x2(acc[1][n / 2], u0, u1);
          g0 = store(t, n, g0, u0, amax);
          if (n + 1 < t.cnt) g1 = store(t, n + 1, g1, u1, amax);
          acc[0][n / 2] = pack_f32x2(g0, g1);
        }
        if (args.half) {
          named_bar_sync(1, 128);
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            if (n >= t.cnt) break;
            float a0, a1;
            unpack_f32x2(acc[0][n / 2], a0, a1);
            quantise(t, n, a0, amax);
            if (n + 1 < t.cnt) quantise(t, n + 1, a1, amax);
          }
        }
      }
    }
  }
  if (total >= 0)
    zero_absent(args, s_offs, (int)blockIdx.x * (C::THREADS / 32) + warp, (int)gridDim.x * (C::THREADS / 32));

  if (S > 1) {
    __syncwarp();
    cluster_sync_all();
    if (warp >= 2 && warp < 6 && ok && first < total) {
      // token n belongs to rank n % S, which adds the S partial sums in rank order
      const Tile t = decode_tile(first, args, s_offs, s_tbase, NT, NG);
      for (int n = rank; n < t.cnt; n += S) {
        float v0 = 0.f, v1 = 0.f;
        for (int c = 0; c < S; ++c) {
          const uint32_t at = sbase + (uint32_t)(n * 256 + wr) * 4u;
          v0 += ld_shared_cluster_f32(at, (uint32_t)c);
          v1 += ld_shared_cluster_f32(at + 512u, (uint32_t)c);
        }
        v0 = store(t, n, v0, v1, s_amax);
        if (args.half) part[n * 256 + wr] = v0;  // (only this thread reads this element of this CTA's)
      }
      if (args.half) {
        named_bar_sync(1, 128);
        for (int n = rank; n < t.cnt; n += S) quantise(t, n, part[n * 256 + wr], s_amax);
      }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();  // the other CTAs have read this one's sums
  } else {
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------------------------
// launches

template <class K>
int configure(K kernel, int smem, std::atomic<int>* configured) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!configured[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return MOE_ERR_CUDA;
    configured[dev].store(1, std::memory_order_release);
  }
  return MOE_OK;
}

int a_map(CUtensorMap* m, const Fp8Gemm& d, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)d.args.K, (cuuint64_t)d.args.a_rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d.args.lda};
  const cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(d.args.A), dims, strides, box, estr,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

int w_map(CUtensorMap* m, const Fp8Gemm& d) {
  const cuuint64_t dims[3] = {(cuuint64_t)d.args.K, (cuuint64_t)d.args.N, (cuuint64_t)d.args.e_count};
  const cuuint64_t strides[2] = {(cuuint64_t)d.ldw, (cuuint64_t)d.w_expert};
  const cuuint32_t box[3] = {(cuuint32_t)BK, 128, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(d.W), dims, strides, box, estr,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

// stores of 32-row boxes, 128 bytes wide (the gate/up form's codes: 64)
int c_map(CUtensorMap* m, const Fp8Gemm& d) {
  const Fp8GemmArgs& a = d.args;
  if (a.half) {
    const cuuint64_t dims[2] = {(cuuint64_t)a.half, (cuuint64_t)a.R};
    const cuuint64_t strides[1] = {(cuuint64_t)a.ld_q};
    const cuuint32_t box[2] = {64, 32};
    const cuuint32_t estr[2] = {1, 1};
    return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.q, dims, strides, box, estr, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  const bool bf16 = a.c_dtype == MOE_DTYPE_BF16;
  const cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.R};
  const cuuint64_t strides[1] = {(cuuint64_t)a.ldc * (bf16 ? 2 : 4)};
  const cuuint32_t box[2] = {bf16 ? 64u : 32u, 32};
  const cuuint32_t estr[2] = {1, 1};
  return encode_tmap(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, a.C, dims,
                     strides, box, estr, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Clusters of S CTAs of a kernel that the device holds at once (they do not cross its groups of SMs, so
// fewer than the CTAs would suggest), asked once for each S.
template <class K>
int resident_clusters(K kernel, int threads, int smem, int S, std::atomic<int> (*known)[9]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][S].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(S);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
  known[dev][S].store(n, std::memory_order_relaxed);
  return n;
}

template <class C>
int launch_wide(const Fp8Gemm& d, int64_t tiles, cudaStream_t st) {
  CUtensorMap am, wm, cm = {};
  int rc = a_map(&am, d, 128);
  if (rc == MOE_OK) rc = w_map(&wm, d);
  if (rc == MOE_OK) rc = c_map(&cm, d);
  if (rc != MOE_OK) return rc;
  static std::atomic<int> configured[64];
  if ((rc = configure(wide_kernel<C>, C::SMEM, configured)) != MOE_OK) return rc;
  if constexpr (C::SPLIT) {
    static std::atomic<int> known[64][9];
    int S = 1;
    for (int t = 2; t <= 4; t *= 2)
      if (tiles <= resident_clusters(wide_kernel<C>, C::THREADS, C::SMEM, t, known)) S = t;
    return launch_pdl_cluster(wide_kernel<C>, dim3((unsigned)(tiles * S)), dim3(C::THREADS), C::SMEM, st, S, am, wm, cm,
                              d.args);
  }
  const int grid = (int)std::min<int64_t>(tiles, device_sm_count());
  return launch_pdl(wide_kernel<C>, dim3(grid), dim3(C::THREADS), C::SMEM, st, am, wm, cm, d.args);
}

template <class C, bool GATHER>
int launch_few(const Fp8Gemm& d, int64_t tiles, cudaStream_t st) {
  CUtensorMap am, wm;
  int rc = a_map(&am, d, GATHER ? 1 : C::NT);
  if (rc == MOE_OK) rc = w_map(&wm, d);
  if (rc != MOE_OK) return rc;
  static std::atomic<int> configured[64];
  if ((rc = configure(few_kernel<C, GATHER>, C::SMEM, configured)) != MOE_OK) return rc;
  // Split k as far as every CTA is still resident at once and keeps two k blocks (one token's gate/up at 64
  // experts, 48 tiles: 11.9 us with one CTA to a tile, 9.4 with four; at 160 experts, 96 tiles: 27.5 with one,
  // 25.6 with two, 31.9 with four, which no longer fit; clusters that share several tiles in turn wait for
  // each other's sums at every one, 64 tokens' down product 269 us against 182).  The query counts one CTA of
  // these kernels per SM whatever they use; PER_SM of them run (192 tiles of two CTAs per SM take 41 us, one
  // and a third rounds of one per SM 49).
  const int KB = (d.args.K + BK - 1) / BK;
  int S = 1;
  static std::atomic<int> known[64][9];
  for (int t = 2; t <= 8 && 2 * t <= KB; ++t)
    if (tiles <= C::PER_SM * resident_clusters(few_kernel<C, GATHER>, C::THREADS, C::SMEM, t, known)) S = t;
  const int64_t grid = S > 1 ? tiles * S : std::min<int64_t>(tiles, device_sm_count() * C::PER_SM);
  return launch_pdl_cluster(few_kernel<C, GATHER>, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, st, S, am, wm,
                            d.args);
}

// Upper bound of the number of token tiles of BT rows: experts with rows plus their full tiles.
int64_t token_tiles(const Fp8Gemm& d, int BT) {
  const Fp8GemmArgs& a = d.args;
  if (a.offsets == nullptr) return tiles_of_rows(a.R, BT);
  return std::min<int64_t>(a.R, std::min<int64_t>(a.R, a.e_count) + a.R / BT);
}

template <bool GATHER>
int launch(const Fp8Gemm& d, cudaStream_t st) {
  const Fp8GemmArgs& a = d.args;
  const int groups = a.offsets == nullptr ? 1 : std::min(a.E, a.R);
  const double rows = (double)a.R / groups;  // per expert, on average
  const int64_t ng2 = a.half ? a.half / 128 : (a.N + 255) / 256;
  const int64_t tt = token_tiles(d, 128);
  const int64_t wide_tiles = a.half ? tt * ng2 : tt * ((a.N + 127) / 128);
  // Few rows per expert: the few-row kernel up to 8 (at 64 experts the down product of 64 tokens, 8 rows,
  // takes 21.2 us against the wide kernel's 24.0 and gate/up 40.5 against 41.0; at 160 experts gate/up of 64
  // tokens, 3.2 rows, 352 against 370, of 256 tokens, 12.8 rows, 391 against 377).  Busier experts among them
  // take several of its tiles, each reading the weights again from L2: routed by a Zipf(1.2) law, 1280 rows
  // over 160 experts take 325 us against 306, 2560 rows 422 against 360.  And up to 128 rows where the
  // wide kernel's tiles would leave half of the SMs idle (64 x 1536 x 5120: 8.2 us against 16.4, with its k
  // split 10.6; 200 rows 14.0 against 11.4 split; gate/up of one expert, 128 rows: 22.9 against 23.8, 200
  // rows 33.6 against 23.9).  32 token rows to a tile from 33 rows on (64 rows: 8.2 us against 8.7 with 16;
  // 32 rows: 8.0 against 7.0).
  const bool idle = 2 * wide_tiles <= device_sm_count();
  if (rows <= 8 || (rows <= 128 && idle)) {
    if (rows <= 32) return launch_few<FewCfg<16, 3, 2>, GATHER>(d, token_tiles(d, 16) * ng2, st);
    return launch_few<FewCfg<32, 5, 1>, GATHER>(d, token_tiles(d, 32) * ng2, st);
  }
  // The plain form's k blocks shared by a cluster where tiles leave half of the SMs idle and are long: from 18 k
  // blocks on, where both cluster sizes cross the time of a CTA alone.  Four CTAs to a tile (333 x 1536): K =
  // 2176 9.46 us against 9.40, 2304 9.46 against 9.74, 2944 9.86 against 11.29, 5120 11.5 against 16.9; two
  // (1100 x 1024): 2176 9.85 against 9.58, 2304 9.92 against 9.92, 2944 10.9 against 11.6.  (Very few tiles
  // cross earlier: 140 x 256, K = 2048 8.17 against 8.93, 1536 7.86 against 7.70.)
  if (!a.half && idle && a.K > 17 * BK) return launch_wide<WideCfg<1, GATHER, false, true>>(d, wide_tiles, st);
  if (a.half) return launch_wide<WideCfg<2, GATHER, true>>(d, tt * ng2, st);
  // 128 weight rows to a tile where tiles of 256 would not fill the SMs
  if (tt * ng2 < device_sm_count()) return launch_wide<WideCfg<1, GATHER, false>>(d, tt * ((a.N + 127) / 128), st);
  return launch_wide<WideCfg<2, GATHER, false>>(d, tt * ng2, st);
}

}  // namespace f8

int fp8_gemm_launch(const Fp8Gemm& d, cudaStream_t st) {
  if (device_sm_count() <= 0) return MOE_ERR_CUDA;
  return d.args.gather != nullptr ? f8::launch<true>(d, st) : f8::launch<false>(d, st);
}

}  // namespace moe
