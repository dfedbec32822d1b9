// The kernels that run the pieces of a shared-prefix attention call.
#pragma once

#include <cuda_runtime.h>

#include "paged.h"

namespace dbsa {

// Tile sizes and CTA count of the kernel that runs a configuration.
struct AttendShape {
  int32_t tile_rows, tile_keys, n_ctas;
};
AttendShape attend_shape(const dbsa_config *cfg);
cudaError_t launch_attend_pieces(const AttendArgs &a, int head_dim, bool f32, cudaStream_t st);

}  // namespace dbsa
