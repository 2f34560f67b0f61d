// Tensor maps of the kernels over a paged cache.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace jfa {

// [rows, cols] of elem_bytes 1 or 2, read in boxes of box_rows x box_cols whose rows are 64 or
// 128 bytes (swizzled by as much); elements outside read as zeros.
bool make_rows_map(CUtensorMap* map, const void* base, int elem_bytes, int64_t rows, int cols, int box_cols,
                   int box_rows);

}  // namespace jfa
