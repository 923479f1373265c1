// few_fp8.cu -- the few-token layer (few.cuh) of experts in block-scaled FP8.
//
// Rows and activations are quantised to E4M3, 128 columns to a scale.  As in the few-row product (fp8_gemm.cu) a k block
// of 128 makes an accumulator by itself, which is scaled by the row's and the weight's scale on its way to FP32 registers.

#include "few.cuh"

namespace moe {
namespace few {

MOE_DEV void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], "
      "[%5], %6;" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

struct Fp8 {
  static constexpr int KB = BK, G = KB, LANE = 4, LEAST = 4, BLOCK_BYTES = KB;
  static constexpr int STAGE = 2 * BLK + NT * BK, TMEM_COLS = ND * 2 * NT;
  static constexpr int WEIGHT_ARRIVALS = 1, FULL_ARRIVALS = WEIGHT_ARRIVALS + 32;

  struct Maps {
    CUtensorMap w[4];  // gate/up, down; the shared expert's
  };
  MOE_DEV static void prefetch(const FewArgs& a, const Maps& maps) {
    if (lane_id() < (a.Is > 0 ? 4 : 2)) prefetch_tmap(&maps.w[lane_id()]);
  }
  MOE_DEV static bool held(const FewArgs& a, int e) { return e >= a.first && e < a.first + a.count; }
  MOE_DEV static int accumulators(int) { return ND; }

  // Distance of an activation row's scales: rows share no 128 bytes, so that an SM whose L1 has one row's does not
  // have another's from before they were made.
  __host__ __device__ static constexpr int scale_pitch(int blocks) { return (blocks + 31) / 32 * 32; }

  MOE_DEV static void write_block(const float (&v)[4], uint8_t* codes, float* scales, int row, int kb, int blocks, int pitch) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3]))));
    float scale, by;
    fp8_scale(m, scale, by);
    reinterpret_cast<uint32_t*>(codes + ((size_t)row * blocks + kb) * KB)[lane_id()] =
        pack_e4m3x4(v[0] * by, v[1] * by, v[2] * by, v[3] * by);
    if (lane_id() == 0) scales[(size_t)row * pitch + kb] = scale;
  }

  struct Weights {
    const CUtensorMap* map;
    int e, row0, row1;
    uint64_t policy;
    MOE_DEV Weights(const FewArgs& a, const Maps& maps, const Unit& un) : policy(streaming_policy()) {
      const bool down = un.flags & DOWN, is_shared = un.flags & SHARED;
      map = &maps.w[(is_shared ? 2 : 0) + (down ? 1 : 0)];
      e = is_shared ? 0 : un.expert;
      row0 = un.place * (down ? 256 : 128);
      row1 = row0 + (down ? 128 : is_shared ? a.Is : a.I);
    }
    MOE_DEV void load(int kb, uint32_t at, uint32_t full) const {
      if (elect_one()) {
        mbar_arrive_expect_tx(full, 2 * BLK);  // (rows past the weight's come as zeros)
        tma_load_3d(at, map, kb * BK, row0, e, full, policy);
        tma_load_3d(at + BLK, map, kb * BK, row1, e, full, policy);
      }
      __syncwarp();
    }
  };

  // A stage's rows of 128 bytes, as the MMA takes them (128-byte swizzle), and the scales.
  struct Rows {
    const FewArgs& a_;
    const uint8_t* src[NT / 4];
    const float* sc;
    int64_t step;
    MOE_DEV Rows(const FewArgs& a, const Maps&, const Unit&) : a_(a) {}
    MOE_DEV void start(const Smem& s, const Unit& un) {
      const FewArgs& a = a_;
      const int lane = lane_id(), piece = lane & 7;
      const bool down = un.flags & DOWN, is_shared = un.flags & SHARED;
      const int inter = is_shared ? a.Is : a.I, groups = (down ? inter : a.H) / G;
      // rows of the unit's tokens (past the last one: that one's again, whose sums are not stored)
      auto row = [&](int c) {
        const int p = un.first + min(c, un.m - 1);
        return !down ? (int)s.token[p] : is_shared ? p - a.T * a.k : p;
      };
      const uint8_t* codes = !down ? a.x_codes : is_shared ? a.act_codes_shared : a.act_codes;
      const int64_t ld = !down ? a.x_ld : inter;
#pragma unroll
      for (int c = 0; c < NT / 4; ++c) src[c] = codes + row(4 * c + (lane >> 3)) * ld + un.kb0 * BK + piece * 16;
      // lanes 0-15: the rows' scales, 16 and 17: the weight's blocks'
      step = 1;
      if (lane < NT) {
        sc = !down ? a.x_scales + row(lane) * a.x_s_row + un.kb0 * a.x_s_grp
                   : (is_shared ? a.act_scales_shared : a.act_scales) + row(lane) * scale_pitch(groups) + un.kb0;
        if (!down) step = a.x_s_grp;
      } else {
        const int blocks = (down ? a.H : 2 * inter) / G, e = is_shared ? 0 : un.expert;
        const int block = min(un.place * (down ? 2 : 1) + (lane & 1) * (down ? 1 : inter / G), blocks - 1);
        sc = (is_shared ? (down ? a.w8s[1].s : a.w8s[0].s) : down ? a.w8[1].s : a.w8[0].s) +
             ((size_t)e * blocks + block) * groups + un.kb0;
      }
    }
    MOE_DEV void load(const Smem&, const Unit& un, int, uint32_t at, float* scales, uint32_t full) {
      const int lane = lane_id(), piece = lane & 7;
#pragma unroll
      for (int c = 0; c < NT / 4; ++c) {
        const int r = 4 * c + (lane >> 3);
        if (4 * c < un.m) cp_async16(at + 2 * BLK + r * 128 + ((piece ^ (r & 7)) << 4), src[c], 16);
        src[c] += BK;
      }
      if (lane < NT + 2) cp_async4(smem_u32(scales + lane), sc);
      sc += step;
      cp_async_arrive(full);
    }
  };

  MOE_DEV static void multiply(uint32_t tmem, int db, uint32_t at, int, int) {
    constexpr uint32_t idesc = make_idesc_e4m3(128, NT);
    const uint64_t rows = make_sdesc_sw128(at + 2 * BLK);
    mma4_e4m3_ss(tmem + (uint32_t)(db * 2 * NT), make_sdesc_sw128(at), rows, idesc);
    mma4_e4m3_ss(tmem + (uint32_t)(db * 2 * NT + NT), make_sdesc_sw128(at + BLK), rows, idesc);
  }

  MOE_DEV static void add(uint64_t (&acc)[2][NT / 2], uint32_t lane_base, int db, const float* f, int, int, uint32_t d_empty) {
    uint32_t v[2][16];
    tmem_ld_32x32b_x16(lane_base + (uint32_t)(db * 2 * NT), v[0]);
    tmem_ld_32x32b_x16(lane_base + (uint32_t)(db * 2 * NT + NT), v[1]);
    uint64_t sa[NT / 2];  // of tokens 2 j and 2 j + 1
#pragma unroll
    for (int j = 0; j < NT / 4; ++j) {
      const ulonglong2 u = reinterpret_cast<const ulonglong2*>(f)[j];
      sa[2 * j] = u.x;
      sa[2 * j + 1] = u.y;
    }
    const uint64_t sw[2] = {pack_f32x2(f[NT], f[NT]), pack_f32x2(f[NT + 1], f[NT + 1])};
    tmem_wait_ld_regs(v[0]);
    tmem_wait_ld_regs(v[1]);
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(d_empty);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) fma_f32x2(acc[h][j], v[h][2 * j], v[h][2 * j + 1], mul_f32x2(sa[j], sw[h]));
  }

  MOE_DEV static float output_scale(const FewArgs&, const Unit&) { return 1.f; }
};

// An FP8 weight [experts][N, K]: boxes of 128 rows and one k block.
int weight_map(CUtensorMap* map, const FewFp8Weight& w, int N, int K, int count) {
  const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)count};
  const cuuint64_t strides[2] = {(cuuint64_t)w.ld, (cuuint64_t)(count > 1 ? w.expert_stride : w.ld * (int64_t)N)};
  const cuuint32_t box[3] = {BK, 128, 1}, one[3] = {1, 1, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(w.q), dims, strides, box, one,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace few

FewLayout few_fp8_layout(int T, int H, int I, int Is, int E, int k) { return few::layout<few::Fp8>(T, H, I, Is, E, k); }

int few_fp8_launch(FewArgs& a, const FewLayout& l, void* ws, cudaStream_t st) {
  few::place(a, l, ws);
  if (a.rows_q != nullptr) {
    a.x_made = nullptr;
    a.x_codes = a.rows_q;
    a.x_ld = a.rows_ld;
    a.x_scales = a.rows_s;
    a.x_s_row = a.rows_s_row;
    a.x_s_grp = a.rows_s_grp;
  } else {
    a.x_codes = a.x_made;
    a.x_ld = a.H;
    a.x_scales = a.x_scales_made;
    a.x_s_row = a.H / few::Fp8::G;
    a.x_s_grp = 1;
  }
  few::Fp8::Maps maps = {};
  int rc = few::weight_map(&maps.w[0], a.w8[0], 2 * a.I, a.H, a.count);
  if (rc == MOE_OK) rc = few::weight_map(&maps.w[1], a.w8[1], a.H, a.I, a.count);
  if (rc == MOE_OK && a.Is > 0) rc = few::weight_map(&maps.w[2], a.w8s[0], 2 * a.Is, a.H, 1);
  if (rc == MOE_OK && a.Is > 0) rc = few::weight_map(&maps.w[3], a.w8s[1], a.H, a.Is, 1);
  return rc == MOE_OK ? few::launch<few::Fp8>(a, maps, st) : rc;
}

}  // namespace moe
