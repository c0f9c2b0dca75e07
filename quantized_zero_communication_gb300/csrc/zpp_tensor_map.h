// zpp_tensor_map.h -- host side of the tensor copies: descriptors of row-major matrices, read in boxes
// of 128 bytes by up to 256 rows with the 128-byte swizzle.
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stdint.h>

namespace zpp {

// `inner` elements of `size` bytes (1: bytes, 2: fp16) in a row, rows `stride` bytes apart (a
// multiple of 16), `rows` of them, in `count` matrices `apart` bytes apart (count 0: a matrix alone, two
// coordinates). `at` is 16-byte aligned; a box has `box_rows` <= 256 rows of 128 bytes.
cudaError_t make_tensor_map(CUtensorMap* map, const void* at, int size, int64_t inner, int64_t rows,
                            int64_t stride, int64_t count, int64_t apart, int box_rows);

}  // namespace zpp
