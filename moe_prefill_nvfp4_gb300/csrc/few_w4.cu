// few_w4.cu -- the few-token layer (few.cuh) of experts in NVFP4.
//
// The weights go to the tensor cores as they lie in memory: packed E2M1 codes with an E4M3 scale to 16 columns are the
// A operand of the block-scaled MMA.  Its B operand is in the same format, so a row of activations becomes six rows of
// E2M1 codes: with s a power of two such that the 16 columns' largest magnitude is at most 6 s,
//   v / s = p1 + 2^-2 p2 + 2^-5 p3 + 2^-8 p4 + 2^-11 p5 + 2^-14 p6 + r,   |r| <= 2^-15.
// (p1 is v / s rounded to E2M1 and off by at most 1; four times that is at most 4, where E2M1 is off by at most 1/2;
// from there on eight times the rest is at most 4.)  So a column is off by at most 2^-15 s, 2^-16.5 of the largest of
// its 16, and a BF16 value within 2^-7 of that one is exact.  The six rows have the same scales and make six columns
// of the accumulator, which the epilogue adds up, smallest first.  s is an E4M3 number of exponent -6 .. 8 times a
// power of two to the row's block of 256 columns, its factor: columns in which the scale would be smaller are
// off by at most 2^-15 2^-6, 2^-30 of the block's largest.  The largest magnitude counts as 2^-115 at least: what is
// smaller is off by at most 2^-15 2^-118.
// A block with a value that is not finite has the factor NaN.  (The MMA knows no sign of a scale: NVFP4 has none.)
//
// Compared with converting the weights to 16 bits in registers this leaves all of an SM's issue slots and
// shared memory bandwidth to the copies: 16 tokens at 160 experts took 294 us with mma.sync on converted weights.

#include "few.cuh"

namespace moe {
namespace few {

MOE_DEV void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[12]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
MOE_DEV void tmem_ld_32x32b_x4(uint32_t taddr, uint32_t (&r)[12]) {  // into the last four
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11])
               : "r"(taddr)
               : "memory");
}

// Loads that are issued where they stand, a block ahead of their use: the compiler would move plain ones down to that, with
// 16 tokens in 230 us instead of 200.  Of what no kernel writes meanwhile, and of what other SMs have stored.
MOE_DEV uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
MOE_DEV uint4 load_l2(const void* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
MOE_DEV float load_l2_f32(const void* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

MOE_DEV void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 32 rows of 16 bytes of shared memory to four columns of tensor memory, for each of its four quarters of lanes.
MOE_DEV void tmem_copy_scales(uint32_t taddr, uint32_t at) {
  const uint64_t desc = (uint64_t)((at & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

MOE_DEV void mma_nvfp4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t scales_a, uint32_t scales_b, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(scales_a), "r"(scales_b), "r"((int)add)
      : "memory");
}

// E2M1 (1) x E2M1 with E4M3 scales (bit 23 = 0), both K-major, N >> 3 at 17, M >> 4 at 24
__host__ __device__ constexpr uint32_t make_idesc_nvfp4(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Eight floats to E2M1 codes, the first in the lowest bits.
MOE_DEV uint32_t pack_e2m1x8(const float (&v)[8]) {
  uint32_t out;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(out)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return out;
}

MOE_DEV void tma_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], "
      "%5;" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}

MOE_DEV void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int u, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
      : "memory");
}

struct W4 {
  static constexpr int KB = 256, LANE = 8, LEAST = 2;
  static constexpr int PIECES = 6, RB = 128;  // rows of codes to an activation row, bytes of one in a k block
  // a block of a row: the pieces, 16 scales, the factor; padded to whole lines
  static constexpr int BLOCK_BYTES = 896, SCALES = PIECES * RB, FACTOR = SCALES + 16;
  // a stage: 256 weight rows, the pieces' rows, the weight's scales, the pieces'.  Scales are as the MMA wants them:
  // of 128 rows and 64 columns 512 bytes, four scales of row r at r % 32 * 16 + r / 32 * 4.
  static constexpr int MAX_N = NT * PIECES, SF = 512, ROWS = 2 * BLK, SCALES_A = ROWS + MAX_N * RB,
                       SCALES_B = SCALES_A + 8 * SF, STAGE = SCALES_B + 4 * SF;
  static constexpr int TMEM_COLS = 256, TMEM_SCALES = 208;  // (32 columns of the weight's scales, 16 of the pieces')
  static constexpr int WEIGHT_ARRIVALS = 2, FULL_ARRIVALS = WEIGHT_ARRIVALS + 1;
  static_assert(STAGE % 1024 == 0 && 2 * MAX_N <= TMEM_SCALES && MAX_N <= 128, "");

  struct Maps {
    CUtensorMap x, act;  // rows of 128 bytes, pieces, blocks, rows of activations
  };
  MOE_DEV static void prefetch(const FewArgs&, const Maps& maps) {
    if (lane_id() < 2) prefetch_tmap(lane_id() == 0 ? &maps.x : &maps.act);
  }
  MOE_DEV static bool held(const FewArgs& a, int e) { return a.w4[0].packed[e] != nullptr && a.w4[1].packed[e] != nullptr; }
  // Columns of an accumulator's half of 128 weight rows; as many accumulators as fit.
  MOE_DEV static int columns(int m) { return (m * PIECES + 15) / 16 * 16; }
  MOE_DEV static int accumulators(int most) { return min(ND, TMEM_SCALES / (2 * columns(most))); }

  __host__ __device__ static constexpr int scale_pitch(int blocks) { return blocks; }

  MOE_DEV static void write_block(const float (&v)[8], uint8_t* rows, float*, int row, int kb, int blocks, int) {
    const int lane = lane_id();
    uint8_t* to = rows + ((size_t)row * blocks + kb) * BLOCK_BYTES;
    // the exponent of the power of two whose sixfold a magnitude does not pass
    auto exponent = [](uint32_t bits) { return (int)(bits >> 23) - 129 + ((bits & 0x7FFFFFu) > 0x400000u); };
    uint32_t most = 0x06000000u;  // 2^-115: the factor is no less than 2^-126
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, abs_bits(v[j]));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    const uint32_t all = __reduce_max_sync(0xffffffffu, most);
    const int top = exponent(all) - 8, code = max(exponent(most) - top, -6);
    const float by = __uint_as_float((uint32_t)(127 - (code + top)) << 23);
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) rest[j] = v[j] * by;
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const uint32_t w = pack_e2m1x8(rest);
      reinterpret_cast<uint32_t*>(to + p * RB)[lane] = w;
      uint32_t h[4];
      e2m1x8_to_f16x2(w, h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        rest[2 * j] = (rest[2 * j] - f.x) * (p == 0 ? 4.f : 8.f);
        rest[2 * j + 1] = (rest[2 * j + 1] - f.y) * (p == 0 ? 4.f : 8.f);
      }
    }
    if (lane % 2 == 0) to[SCALES + lane / 2] = (uint8_t)((code + 7) << 3);
    if (lane == 0)
      *reinterpret_cast<float*>(to + FACTOR) = __uint_as_float(all < 0x7F800000u ? (uint32_t)(127 + top) << 23 : 0x7FC00000u);
  }

  struct Weights {
    const uint8_t* map;
    int row0, row1, scale_pitch, end;
    uint64_t policy;
    const uint8_t* scales[2];  // this lane's, one of 32 rows, of the rows' two halves
    uint4 v[2][4];
    MOE_DEV Weights(const FewArgs& a, const Maps&, const Unit& un) : end(un.kb1), policy(streaming_policy()) {
      const bool down = un.flags & DOWN;
      const FewW4Weight& w = a.w4[down ? 1 : 0];
      map = static_cast<const uint8_t*>(w.maps) + (size_t)un.expert * 2 * sizeof(CUtensorMap);
      row0 = un.place * (down ? 256 : 128);
      row1 = row0 + (down ? 128 : a.I);
      scale_pitch = (down ? a.I : a.H) / 16;
      const uint8_t* of = static_cast<const uint8_t*>(w.scales[un.expert]);
      scales[0] = of + (size_t)(row0 + lane_id()) * scale_pitch;
      scales[1] = of + (size_t)(row1 + lane_id()) * scale_pitch;
      fetch_scales(un.kb0);
    }
    // A block's 16 scales of four rows of each half to a lane, and from there to where the MMA wants them.  (As copies
    // of 4 bytes past the registers they took 3 us more of 48, one token, and 5 of 209, 16 tokens.)
    MOE_DEV void fetch_scales(int kb) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[h][j] = load_once(scales[h] + (size_t)(32 * j) * scale_pitch + kb * 16);
    }
    MOE_DEV void store_scales(uint32_t at, uint32_t full) const {
      const uint32_t to = at + SCALES_A + lane_id() * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 (&w)[4] = v[h];
        sts128(to + (h * 4 + 0) * SF, w[0].x, w[1].x, w[2].x, w[3].x);
        sts128(to + (h * 4 + 1) * SF, w[0].y, w[1].y, w[2].y, w[3].y);
        sts128(to + (h * 4 + 2) * SF, w[0].z, w[1].z, w[2].z, w[3].z);
        sts128(to + (h * 4 + 3) * SF, w[0].w, w[1].w, w[2].w, w[3].w);
      }
      __syncwarp();
      if (lane_id() == 0) mbar_arrive(full);
    }
    MOE_DEV void load(int kb, uint32_t at, uint32_t full) {
      if (elect_one()) {
        mbar_arrive_expect_tx(full, 2 * BLK);
        tma_load_2d(at, map, kb * RB, row0, full, policy);
        tma_load_2d(at + BLK, map, kb * RB, row1, full, policy);
      }
      __syncwarp();
      store_scales(at, full);
      if (kb + 1 < end) fetch_scales(kb + 1);
    }
  };

  // A token's six rows are one tile; their scales and the factor go through registers, a block ahead.
  struct Rows {
    const uint8_t* of;
    const CUtensorMap* map;
    size_t pitch;
    uint4 v[MAX_N / 32];  // the block's scales of rows lane, lane + 32, ...
    float factor;         // of token `lane`
    MOE_DEV Rows(const FewArgs& a, const Maps& maps, const Unit& un) {
      const bool down = un.flags & DOWN;
      pitch = (size_t)((down ? a.I : a.H) / KB) * BLOCK_BYTES;
      of = down ? a.act_codes : a.x_made;
      map = down ? &maps.act : &maps.x;
    }
    MOE_DEV static int row(const Smem& s, const Unit& un, int c) {
      return un.flags & DOWN ? un.first + c : (int)s.token[un.first + c];
    }
    MOE_DEV void start(const Smem& s, const Unit& un) {
      fence_proxy_async_global();  // (the rows were stored through the generic proxy)
      fetch(s, un, un.kb0);
    }
    MOE_DEV void fetch(const Smem& s, const Unit& un, int kb) {
      const int lane = lane_id();
#pragma unroll
      for (int j = 0; j < MAX_N / 32; ++j) {
        const int c = (lane + 32 * j) / PIECES;
        if (c < un.m) v[j] = load_l2(of + row(s, un, c) * pitch + (size_t)kb * BLOCK_BYTES + SCALES);
      }
      if (lane < un.m) factor = load_l2_f32(of + row(s, un, lane) * pitch + (size_t)kb * BLOCK_BYTES + FACTOR);
    }
    MOE_DEV void load(const Smem& s, const Unit& un, int kb, uint32_t at, float* factors, uint32_t full) {
      const int lane = lane_id();
      if (elect_one())
        for (int c = 0; c < un.m; ++c) tma_load_4d(at + ROWS + c * PIECES * RB, map, 0, 0, kb, row(s, un, c), full);
      __syncwarp();
      const uint32_t to = at + SCALES_B + lane * 16;
      sts128(to, v[0].x, v[1].x, v[2].x, 0);
      sts128(to + SF, v[0].y, v[1].y, v[2].y, 0);
      sts128(to + 2 * SF, v[0].z, v[1].z, v[2].z, 0);
      sts128(to + 3 * SF, v[0].w, v[1].w, v[2].w, 0);
      if (lane < un.m) factors[lane] = factor;
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(full, un.m * PIECES * RB);
      if (kb + 1 < un.kb1) fetch(s, un, kb + 1);
    }
  };

  MOE_DEV static void multiply(uint32_t tmem, int db, uint32_t at, int m, int most) {
    const uint32_t idesc = make_idesc_nvfp4(128, columns(m));
    const int half = columns(most);
    const uint64_t rows = make_sdesc_sw128(at + ROWS);
#pragma unroll
    for (int k64 = 0; k64 < 4; ++k64) {
      const uint32_t scales_b = tmem + TMEM_SCALES + 32 + k64 * 4;
      tmem_copy_scales(scales_b, at + SCALES_B + k64 * SF);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t scales_a = tmem + TMEM_SCALES + h * 16 + k64 * 4;
        tmem_copy_scales(scales_a, at + SCALES_A + (h * 4 + k64) * SF);
        mma_nvfp4_ss(tmem + (uint32_t)((2 * db + h) * half), make_sdesc_sw128(at + h * BLK) + k64 * 2, rows + k64 * 2, idesc,
                     scales_a, scales_b, k64 > 0);
      }
    }
  }

  MOE_DEV static void add(uint64_t (&acc)[2][NT / 2], uint32_t lane_base, int db, const float* f, int m, int most,
                          uint32_t d_empty) {
    const int half = columns(most);
    const uint32_t at = lane_base + (uint32_t)(2 * db * half);
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) {
      if (2 * j < m) {  // two tokens at once
        uint32_t v[2][2 * PIECES];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t from = at + (uint32_t)(h * half + j * 2 * PIECES);
          tmem_ld_32x32b_x8(from, v[h]);
          tmem_ld_32x32b_x4(from + 8, v[h]);
        }
        tmem_wait_ld_regs(v[0]);
        tmem_wait_ld_regs(v[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float t[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t* p = v[h] + i * PIECES;
            t[i] = __uint_as_float(p[5]);
#pragma unroll
            for (int q = 4; q > 0; --q) t[i] = __fmaf_rn(t[i], 0.125f, __uint_as_float(p[q]));
            t[i] = __fmaf_rn(t[i], 0.25f, __uint_as_float(p[0]));
          }
          fma_f32x2(acc[h][j], __float_as_uint(t[0]), __float_as_uint(t[1]), pack_f32x2(f[2 * j], f[2 * j + 1]));
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(d_empty);
  }

  MOE_DEV static float output_scale(const FewArgs& a, const Unit& un) {
    return (un.flags & DOWN ? a.w4[1].scale2 : a.w4[0].scale2)[un.expert];
  }
};

// Activations [rows][blocks] of BLOCK_BYTES: tiles of the six pieces of a block.
int rows_map(CUtensorMap* map, const uint8_t* base, int blocks, int rows) {
  const cuuint64_t dims[4] = {W4::RB, W4::PIECES, (cuuint64_t)blocks, (cuuint64_t)rows};
  const cuuint64_t strides[3] = {W4::RB, W4::BLOCK_BYTES, (cuuint64_t)blocks * W4::BLOCK_BYTES};
  const cuuint32_t box[4] = {W4::RB, W4::PIECES, 1, 1}, one[4] = {1, 1, 1, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, one,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace few

FewLayout few_w4_layout(int T, int H, int I, int Is, int E, int k) { return few::layout<few::W4>(T, H, I, Is, E, k); }

int few_w4_launch(FewArgs& a, const FewLayout& l, void* ws, cudaStream_t st) {
  few::place(a, l, ws);
  few::W4::Maps maps = {};
  int rc = few::rows_map(&maps.x, a.x_made, a.H / few::W4::KB, a.T);
  if (rc == MOE_OK) rc = few::rows_map(&maps.act, a.act_codes, a.I / few::W4::KB, a.T * a.k);
  return rc == MOE_OK ? few::launch<few::W4>(a, maps, st) : rc;
}

}  // namespace moe
