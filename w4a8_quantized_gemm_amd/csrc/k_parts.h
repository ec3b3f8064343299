// How the 16 x 16 tile kernel cuts a row's K-tiles into parts: between workgroups
// (splits) and, within one, between its wave pairs.
#pragma once
#include <hip/hip_runtime.h>

namespace w4a8 {

// First K-tile of part `part` of `parts` of a row of `all` K-tiles (and the end
// of the part before it).
__host__ __device__ inline int k_part_first(int all, int part, int parts) {
    return (int)((long long)all * part / parts);
}

// Last step whose weights a part of `tiles` K-tiles loads; steps behind it load
// the same ones again.  One K-tile in two parts leaves the first part none: its
// waves multiply X tiles of zeros by the weights of the part's first K-tile, which
// lies in the row (part < parts), and never by those in front of it, whose scalar
// offset would leave the array without the buffer's range check noticing.
template <int KIN>
__host__ __device__ inline int k_last_step(int tiles) {
    return KIN == 1 || tiles > 0 ? tiles - 1 : 0;
}

}  // namespace w4a8
