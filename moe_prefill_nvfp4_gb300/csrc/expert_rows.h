// expert_rows.h -- checks and counts over expert offsets, on the host and on the device.
#pragma once

#if defined(__CUDACC__)
#define MOE_HOST_DEV __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEV inline
#endif

namespace moe {

// Whether [lo, hi) can be one expert's of R sorted rows.  Compared, never subtracted: the offsets are device data
// of any value, and hi - lo of a step from 2^30 down to -2^31 wraps to a positive count.  Where every step
// passes, the offsets are a non-decreasing sequence within [0, R].
MOE_HOST_DEV bool expert_rows_ok(int lo, int hi, int R) { return 0 <= lo && lo <= hi && hi <= R; }

// Tiles of `per` rows that hold `rows` >= 0 rows (rows + per - 1 could pass 2^31).
MOE_HOST_DEV int tiles_of_rows(int rows, int per) { return rows > 0 ? 1 + (rows - 1) / per : 0; }

}  // namespace moe
