// The kernels that run the pieces of a shared-prefix attention call.
#pragma once

#include <cuda_runtime.h>

#include "paged.h"

namespace dbsa {

// Tile sizes and CTA count of the kernel that runs a call with `rows` packed rows
// per KV head.
struct AttendShape {
  int32_t tile_rows, tile_keys, n_ctas;
  int32_t min_tile_rows, max_tile_rows;   // over all calls
};
AttendShape attend_shape(const dbsa_config *cfg, int rows, int64_t prefix_len);
cudaError_t launch_attend_pieces(const AttendArgs &a, int head_dim, bool f32, cudaStream_t st);

}  // namespace dbsa
