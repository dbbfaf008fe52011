// route.cuh -- the routing steps that other translation units launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hq_internal.h"

namespace hq {
namespace route {

// Workspace of a sort: a histogram per tile of pairs, if there is more than one
// tile (and 256 bytes in front, since a size of 0 is a bad argument's).
size_t sort_workspace_bytes(long pairs, int E);
int sort_launches(long pairs);
bool sort_supported(long pairs, int E, int align);
cudaError_t launch_sort(const int32_t* ids, int pairs, int E, int align, int32_t* pos, int32_t* offsets,
                        int32_t* counts, void* ws, cudaStream_t st);
// y[t] = sum_j w[t][j] z[pos[t][j]] (w nullptr: plain sums); y of z's type, or
// either of them fp32.
cudaError_t launch_combine(hq_dtype zd, hq_dtype yd, const void* z, const int32_t* pos, const float* w, void* y,
                           int T, int k, int H, int n_rows, cudaStream_t st);

}  // namespace route
}  // namespace hq
