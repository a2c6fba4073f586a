// Index arithmetic of paged rows at the ends of its types (host and device, no CUDA).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SPECV_HD __host__ __device__ __forceinline__
#else
#define SPECV_HD inline
#endif

namespace specv {

// Whether a block table row of `width` entries has entry first + g (first, g >= 0; with pages
// of one token their sum may pass 31 bits).
SPECV_HD bool in_table(int32_t first, int32_t g, int32_t width) {
    return (uint32_t)first + (uint32_t)g < (uint32_t)width;
}

// First entry, of a table row of `width`, behind the pages of `keep` >= 0 tokens.
SPECV_HD int32_t entries_kept(int32_t keep, int32_t page_size, int32_t width) {
    const int64_t n = ((int64_t)keep + page_size - 1) / page_size;
    return n < width ? (int32_t)n : width;
}

// 16-byte pieces of `rows` cached rows of `dim` elements (a multiple of 32) of `elem` bytes: whole
// ones in a row.  (A page may have 2^32 bytes, 2^28 pieces.)
SPECV_HD int32_t row_pieces(int32_t rows, int32_t dim, int32_t elem) { return rows * (dim * elem / 16); }

}  // namespace specv
