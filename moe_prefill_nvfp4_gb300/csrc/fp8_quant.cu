// fp8_quant.cu -- quantisation to E4M3 with one FP32 scale per 128 elements of a row (activations)
// or per 128 x 128 block (weights): the operands of the FP8 products.
//
//   a = max(max |x| over the group, 2^-100),  s = a / 448,  q = e4m3(x * (448 * (1 / a)))
//
// in FP32, each operation correctly rounded; q rounds to nearest even (the product is at most
// 448 (1 + 2^-22), which rounds to 448, so nothing saturates).  The floor of a keeps 448 / a and s
// normal FP32 numbers; a group of zeros gives q = 0.  A group with an infinity or a
// NaN gives s = NaN and codes NaN: whatever reads it is NaN, no finite value stands for it.
//
// Bound by memory: each element is read once (held in registers between the maximum and the
// rounding), its code is written once.  Measured on GB300 (read and written bytes): rows 8192 x 5120 BF16
// 20.8 us, 6.1 TB/s, FP32 32.8 us, 6.4 TB/s; rows on no 16-byte boundary (8192 x 5119 BF16) 27 us, 4.7 TB/s;
// blocks of 16384 x 5120 BF16 40 us, 6.3 TB/s.

#include <algorithm>
#include <atomic>

#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace fq {

constexpr int G = 128;

// Bits of |x| compare like the magnitudes, with inf above every number and NaN above inf, so an
// unsigned maximum keeps what is not finite.
MOE_DEV uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

template <typename T>
MOE_DEV float load1(const T* p);
template <>
MOE_DEV float load1<uint16_t>(const uint16_t* p) {
  return __uint_as_float((uint32_t)__ldg(p) << 16);
}
template <>
MOE_DEV float load1<float>(const float* p) {
  return __ldg(p);
}

// 16 consecutive elements, 16-byte aligned, as they are in memory
template <typename T>
struct Raw16 {
  uint4 w[sizeof(T)];
};
template <typename T>
MOE_DEV Raw16<T> load16(const T* p) {
  Raw16<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) r.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
MOE_DEV void unpack16(const Raw16<uint16_t>& r, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = bf16_lo(w[j]);
      v[8 * i + 2 * j + 1] = bf16_hi(w[j]);
    }
  }
}
MOE_DEV void unpack16(const Raw16<float>& r, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x);
    v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z);
    v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}

// A warp's place in the items (row, one of per_row pieces of it), advanced without divisions.
struct Walk {
  uint32_t row, piece, drow, dpiece, per_row;
  MOE_DEV Walk(uint32_t warps, uint32_t first, uint32_t per) : per_row(per) {
    row = first / per;
    piece = first - row * per;
    drow = warps / per;
    dpiece = warps - drow * per;
  }
  MOE_DEV void next() {
    row += drow;
    piece += dpiece;
    if (piece >= per_row) {
      piece -= per_row;
      ++row;
    }
  }
};

// Rows, 16 elements to a lane and 8 lanes to a group: a warp takes four consecutive groups of one
// row, the next four on their way meanwhile.  For 16-byte aligned rows; K need not be a multiple of 16
// (the last lane's elements are then loaded one by one).
template <typename T>
__global__ void __launch_bounds__(256) rows_vec_kernel(const T* __restrict__ x, int64_t ld_x, int R, int K, uint8_t* q,
                                                       int64_t ld_q, float* s, int64_t s_row, int64_t s_grp) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int sub = lane & 7;
  const int ngrp = (K + G - 1) / G;
  Walk at(gridDim.x * 8, blockIdx.x * 8 + (threadIdx.x >> 5), (ngrp + 3) / 4);
  // this lane's elements of piece p of a row: group, first column, how many
  auto group = [&](uint32_t p) { return (int)p * 4 + (lane >> 3); };
  auto load = [&](const Walk& w, Raw16<T>& r) {
    const int k0 = group(w.piece) * G + sub * 16;
    if (w.row < (uint32_t)R && k0 + 16 <= K) r = load16(x + w.row * ld_x + k0);
  };
  Raw16<T> cur = {}, nxt = {};
  load(at, cur);
  while (at.row < (uint32_t)R) {
    Walk then = at;
    then.next();
    load(then, nxt);
    const int grp = group(at.piece), k0 = grp * G + sub * 16;
    const int n = max(0, min(16, K - k0));
    float v[16];
    unpack16(cur, v);
    if (n < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = i < n ? load1(x + at.row * ld_x + k0 + i) : 0.f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, abs_bits(v[i]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float scale, inv;
    fp8_scale(m, scale, inv);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack_e4m3x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    uint8_t* dst = q + at.row * ld_q + k0;
    if (n == 16) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) dst[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
    if (sub == 0 && grp < ngrp) s[at.row * s_row + grp * s_grp] = scale;
    at = then;
    cur = nxt;
  }
}

// Rows of any alignment, 4 consecutive elements to a lane and a warp to a group: four groups of a row at a
// time, the next four on their way meanwhile.  Codes are stored as words (q is 16-byte aligned with ld_q
// a multiple of 16); the four groups' scales are worked out by a lane each.
//
// The lane's elements are loaded by words: a BF16 row that starts inside one has them in three, of which
// the second half of the last is the row's next element (none is read past the row: `whole`).
template <typename T>
struct Words {
  static constexpr int N = sizeof(T) == 2 ? 3 : 4;
  uint32_t w[4][N];
};

template <typename T>
__global__ void __launch_bounds__(256) rows_any_kernel(const T* __restrict__ x, int64_t ld_x, int R, int K, uint8_t* q,
                                                       int64_t ld_q, float* s, int64_t s_row, int64_t s_grp) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int ngrp = (K + G - 1) / G;
  auto column = [&](const Walk& at, int u) { return ((int)at.piece * 4 + u) * G + lane * 4; };
  auto odd = [&](const Walk& at) {
    return sizeof(T) == 2 ? (int)((reinterpret_cast<uintptr_t>(x + at.row * ld_x) >> 1) & 1) : 0;
  };
  auto load = [&](const Walk& at, Words<T>& r) {
    const int o = odd(at);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = column(at, u);
      const bool whole = at.row < (uint32_t)R && k + 4 + o <= K;
      const uint32_t* p = reinterpret_cast<const uint32_t*>(x + at.row * ld_x + k - o);
#pragma unroll
      for (int i = 0; i < Words<T>::N; ++i)
        r.w[u][i] = whole && (sizeof(T) == 4 || i < 2 || o) ? __ldg(p + i) : 0;
    }
  };
  Walk at(gridDim.x * 8, blockIdx.x * 8 + (threadIdx.x >> 5), (ngrp + 3) / 4);
  Words<T> cur, nxt;
  load(at, cur);
  while (at.row < (uint32_t)R) {
    Walk then = at;
    then.next();
    load(then, nxt);
    const int o = odd(at);
    float v[4][4];
    uint32_t mine = 0;  // of group lane % 4
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = column(at, u);
      if (k + 4 + o <= K) {
        if constexpr (sizeof(T) == 2) {
          const uint32_t lo = o ? __funnelshift_r(cur.w[u][0], cur.w[u][1], 16) : cur.w[u][0];
          const uint32_t hi = o ? __funnelshift_r(cur.w[u][1], cur.w[u][2], 16) : cur.w[u][1];
          v[u][0] = bf16_lo(lo);
          v[u][1] = bf16_hi(lo);
          v[u][2] = bf16_lo(hi);
          v[u][3] = bf16_hi(hi);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] = __uint_as_float(cur.w[u][i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = k + i < K ? load1(x + at.row * ld_x + k + i) : 0.f;
      }
      const uint32_t m = __reduce_max_sync(
          0xffffffffu, max(max(abs_bits(v[u][0]), abs_bits(v[u][1])), max(abs_bits(v[u][2]), abs_bits(v[u][3]))));
      if ((lane & 3) == u) mine = m;
    }
    float scale, inv4;
    fp8_scale(mine, scale, inv4);
    const int grp = (int)at.piece * 4 + lane;
    if (lane < 4 && grp < ngrp) s[at.row * s_row + grp * s_grp] = scale;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float inv = __shfl_sync(0xffffffffu, inv4, u);
      const uint32_t c = pack_e4m3x4(v[u][0] * inv, v[u][1] * inv, v[u][2] * inv, v[u][3] * inv);
      const int k = column(at, u);
      uint8_t* dst = q + at.row * ld_q + k;
      if (k + 4 <= K) {
        *reinterpret_cast<uint32_t*>(dst) = c;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (k + i < K) dst[i] = (uint8_t)(c >> (8 * i));
      }
    }
    at = then;
    cur = nxt;
  }
}

// Weights: a CTA of 256 threads per 128 x 128 block, 64 elements to a thread (lane: 4 consecutive
// columns; warp w: rows w, w + 8, ...).  VEC: 4-element loads (rows 4-element aligned).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 3) blocks_kernel(const T* __restrict__ w, int64_t ld_w, int N, int K, uint8_t* q,
                                                     int64_t ld_q, float* s) {
  __shared__ uint32_t s_max[8];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k0 = blockIdx.x * G + lane * 4;
  const int n0 = blockIdx.y * G + warp;
  float v[16][4];
  uint32_t m = 0;
  if (VEC && (blockIdx.x + 1) * G <= K && (blockIdx.y + 1) * G <= N) {
    // every load before the first use
    uint32_t raw[16][sizeof(T)];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const T* src = w + (int64_t)(n0 + 8 * r) * ld_w + k0;
      if constexpr (sizeof(T) == 2) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(src));
        raw[r][0] = a.x;
        raw[r][1] = a.y;
      } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(src));
        raw[r][0] = a.x;
        raw[r][1] = a.y;
        raw[r][2] = a.z;
        raw[r][3] = a.w;
      }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[r][i] = sizeof(T) == 4 ? __uint_as_float(raw[r][i]) : i & 1 ? bf16_hi(raw[r][i >> 1]) : bf16_lo(raw[r][i >> 1]);
  } else {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int n = n0 + 8 * r;
      const T* src = w + (int64_t)n * ld_w + k0;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[r][i] = n < N && k0 + i < K ? load1(src + i) : 0.f;
    }
  }
#pragma unroll
  for (int r = 0; r < 16; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, abs_bits(v[r][i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  float scale, inv;
  fp8_scale(m, scale, inv);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int n = n0 + 8 * r;
    if (n >= N) break;
    const uint32_t c = pack_e4m3x4(v[r][0] * inv, v[r][1] * inv, v[r][2] * inv, v[r][3] * inv);
    uint8_t* dst = q + (int64_t)n * ld_q + k0;
    if (k0 + 4 <= K) {
      *reinterpret_cast<uint32_t*>(dst) = c;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k0 + i < K) dst[i] = (uint8_t)(c >> (8 * i));
    }
  }
  if (threadIdx.x == 0) s[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = scale;
}

// CTAs of 256 threads of this kernel that one SM holds, asked once.
template <class K>
int per_sm(K kernel, std::atomic<int>& known) {
  int n = known.load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, 256, 0) != cudaSuccess || n < 1) return 1;
  known.store(n, std::memory_order_relaxed);
  return n;
}

template <typename T>
int rows(const T* x, int64_t ld_x, int R, int K, uint8_t* q, int64_t ld_q, float* s, int64_t s_row, int64_t s_grp,
         cudaStream_t st) {
  const int nsm = device_sm_count();
  if (nsm <= 0) return MOE_ERR_CUDA;
  const int ngrp = (K + G - 1) / G;
  const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (ld_x * (int64_t)sizeof(T)) % 16 == 0;
  const int64_t warps = (int64_t)R * ((ngrp + 3) / 4);  // both kernels give a warp four groups
  if (warps >= (1ll << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  static std::atomic<int> vec_per_sm, any_per_sm;
  const int fit = vec ? per_sm(rows_vec_kernel<T>, vec_per_sm) : per_sm(rows_any_kernel<T>, any_per_sm);
  const int grid = (int)std::min<int64_t>((warps + 7) / 8, (int64_t)nsm * fit);
  return vec ? launch_pdl(rows_vec_kernel<T>, dim3(grid), dim3(256), 0, st, x, ld_x, R, K, q, ld_q, s, s_row, s_grp)
             : launch_pdl(rows_any_kernel<T>, dim3(grid), dim3(256), 0, st, x, ld_x, R, K, q, ld_q, s, s_row, s_grp);
}

template <typename T>
int blocks(const T* w, int64_t ld_w, int N, int K, uint8_t* q, int64_t ld_q, float* s, cudaStream_t st) {
  const dim3 grid((K + G - 1) / G, (N + G - 1) / G);
  const bool vec = reinterpret_cast<uintptr_t>(w) % (4 * sizeof(T)) == 0 && ld_w % 4 == 0;
  return vec ? launch_pdl(blocks_kernel<T, true>, grid, dim3(256), 0, st, w, ld_w, N, K, q, ld_q, s)
             : launch_pdl(blocks_kernel<T, false>, grid, dim3(256), 0, st, w, ld_w, N, K, q, ld_q, s);
}

}  // namespace fq

int fp8_quantize_rows_launch(const void* x, int x_dtype, int64_t ld_x, int R, int K, uint8_t* q, int64_t ld_q, float* s,
                             int64_t s_row, int64_t s_grp, cudaStream_t st) {
  return x_dtype == MOE_DTYPE_BF16
             ? fq::rows(static_cast<const uint16_t*>(x), ld_x, R, K, q, ld_q, s, s_row, s_grp, st)
             : fq::rows(static_cast<const float*>(x), ld_x, R, K, q, ld_q, s, s_row, s_grp, st);
}

int fp8_quantize_blocks_launch(const void* w, int w_dtype, int64_t ld_w, int N, int K, uint8_t* q, int64_t ld_q,
                               float* s, cudaStream_t st) {
  return w_dtype == MOE_DTYPE_BF16 ? fq::blocks(static_cast<const uint16_t*>(w), ld_w, N, K, q, ld_q, s, st)
                                   : fq::blocks(static_cast<const float*>(w), ld_w, N, K, q, ld_q, s, st);
}

}  // namespace moe
