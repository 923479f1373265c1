// few.h -- arguments of the few-token layers (few.cuh).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

struct FewFp8Weight {  // codes [experts][N, ld], scales [experts][N / 128][K / 128]
  const uint8_t* q;
  int64_t ld, expert_stride;
  const float* s;
};
struct FewW4Weight {  // by expert (an expert table's arrays)
  const void* maps;           // two tensor maps each: boxes of 128 rows and 128 bytes of the packed codes, and another
  const void* const* packed;  // (NULL: absent)
  const void* const* scales;
  const float* scale2;
};

struct FewArgs {
  const uint16_t* x;         // BF16 [T, H]
  const uint8_t* rows_q;     // FP8: NULL, or the rows' codes and scales (x is then the router's only)
  const float* rows_s;
  int64_t rows_ld, rows_s_row, rows_s_grp;
  const uint16_t* w_router;  // [E, H], or
  const float* logits;       // [T, E] (the other is NULL)
  const float* bias;         // [E] or NULL
  int T, H, I, Is, E, k;     // Is: the shared expert's intermediate size, 0 without
  int first, count;          // the experts held here
  int renormalize;
  float routed_scale, limit, shared_limit;
  FewFp8Weight w8[2], w8s[2];  // gate/up and down; the shared expert's
  FewW4Weight w4[2];
  const uint16_t* shared_out;  // NULL, or BF16 [T, H] to add
  uint16_t* out;               // BF16 [T, H]
  int* err;
  uint64_t wait_ns;            // bound of every wait
  // workspace
  int *counters, *ready, *block_done, *columns_done;
  int n_counters, blocks_max;
  int slices[2], slice_blocks[2];  // of k, gate/up and down
  size_t y_slice;
  float* logits_ws;
  const uint8_t* x_codes;  // the tokens' rows: the given ones, or
  const float* x_scales;
  int64_t x_ld, x_s_row, x_s_grp;
  uint8_t* x_made;         // these, made of x (NULL: given)
  float* x_scales_made;
  uint8_t *act_codes, *act_codes_shared;
  float *gu, *act_scales, *gu_shared, *act_scales_shared, *Y;
};

struct FewLayout {
  size_t counters, logits, x_values, x_scales, gu, act_values, act_scales, gu_shared, act_values_shared, act_scales_shared, Y,
      total;
  size_t y_slice;
  int n_counters, n_ready, n_blocks, n_columns, blocks_max;
  int slices[2], slice_blocks[2];
};
FewLayout few_fp8_layout(int T, int H, int I, int Is, int E, int k);
int few_fp8_launch(FewArgs& a, const FewLayout& l, void* ws, cudaStream_t st);
FewLayout few_w4_layout(int T, int H, int I, int Is, int E, int k);
int few_w4_launch(FewArgs& a, const FewLayout& l, void* ws, cudaStream_t st);

}  // namespace moe
