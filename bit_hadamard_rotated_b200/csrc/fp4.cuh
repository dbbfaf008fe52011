// fp4.cuh -- what the microscaled 4-bit floating-point kernels share: the
// scale tile's layout and the host-side checks and launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hq_internal.h"

namespace hq {
namespace fp4 {

// Scales lie in tiles of 128 rows x 4 scales, 512 bytes: the byte of row r,
// scale j of the tile at (r % 32) * 16 + (r / 32) * 4 + j, the order in which
// tcgen05.cp puts a tile into four tensor-memory columns (lane r % 32, column
// r / 32, one 32-bit word of four scales).  Tiles of one row block follow one
// another along K, row blocks after that.

// Values of K under one tile.
__host__ __device__ constexpr int tile_k(int fmt) { return fmt == HQ_FP4_NV ? 64 : 128; }
// Scale tiles along K.
__host__ __device__ constexpr int scale_tiles(int fmt, int K) { return (K + tile_k(fmt) - 1) / tile_k(fmt); }
// Byte offset of the 4-scale cell of a row in tile kt of kb along K.
__host__ __device__ constexpr size_t scale_cell(long row, int kt, int kb) {
  return (static_cast<size_t>(row >> 7) * kb + kt) * 512 + (row & 31) * 16 + (row >> 5 & 3) * 4;
}
constexpr size_t scale_bytes(int fmt, long rows, int K) {
  return static_cast<size_t>((rows + 127) / 128) * scale_tiles(fmt, K) * 512;
}

hq_status check_rows(const void* x, hq_dtype xd, size_t ldx, int K);
hq_status check_shape(int fmt, long rows, int K);
hq_status check_matrix(const hq_fp4_matrix* m);

// Quantises `rows` rows of x.  pos == nullptr: row r to row r, with the scale
// tiles' padding rows zeroed and, if asked for, the rounded values written.
// Otherwise row r goes to each of its k rows pos[r][j] that lie in
// [0, dst_rows); the other rows of codes and scales are left as they are.
cudaError_t launch_quantize(int fmt, hq_dtype xd, const void* x, size_t ldx, int rows, int K, const float* ts,
                            uint8_t* codes, uint8_t* scales, void* values, const int32_t* pos, int k,
                            int dst_rows, cudaStream_t st);

}  // namespace fp4
}  // namespace hq
