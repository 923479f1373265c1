// few.h -- arguments of the few-token layers (few_tokens.cu).
#pragma once

#include <cuda.h>
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
  const void* const* packed;
  const CUtensorMap* maps;  // [E][2]: packed weights (16 rows x 4 lines of 128 bytes), scales (16 rows x 64 bytes)
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
  // workspace
  int *counters, *ready, *group_done, *tile_done;
  int n_counters, groups_max;
  float* logits_ws;
  uint8_t *x_rec, *act_rec, *act_rec_shared;
  float *act, *act_shared, *Y;
};

struct FewLayout {
  size_t counters, logits, x_rec, act, act_shared, act_rec, act_rec_shared, Y, total;
  int n_counters, n_ready, n_groups, n_tiles, groups_max;
};
FewLayout few_layout(bool w4, int T, int H, int I, int Is, int E, int k);
int few_launch(bool w4, FewArgs& a, const FewLayout& l, void* ws, cudaStream_t st);

}  // namespace moe
