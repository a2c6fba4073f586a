// How the library's workspace grows (host only, no CUDA).
#pragma once

#include <stddef.h>

namespace specv {

// Allocates a buffer of at least `need` bytes in the place of one of `have` that
// was outgrown but stays allocated.  At least twice the old size, so that the
// outgrown buffers together stay below the current one, and 64 MB; where that
// much cannot be had, `need` itself.  alloc(bytes) says whether it could; returns
// the bytes allocated, 0 for none.
template <typename Alloc> size_t grow_buffer(size_t need, size_t have, Alloc alloc) {
    size_t want = (size_t)64 << 20;
    if (want < need) want = need;
    if (want < 2 * have) want = 2 * have;
    if (alloc(want)) return want;
    return want > need && alloc(need) ? need : 0;
}

}  // namespace specv
