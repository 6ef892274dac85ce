// Which 16-byte units of a row the layer norm kernels (srnl_norm.cu) read whole.  Plain C++: the
// kernels and the host see the same rule.
#pragma once

#include <climits>
#include <cstdint>

#ifdef __CUDACC__
#define SRNL_NORM_FN __host__ __device__ __forceinline__
#else
#define SRNL_NORM_FN inline
#endif

namespace srnl {

// Values from the start of row r to the end of a buffer of `rows` rows, or INT_MAX where that is more
// than a unit's length behind the row in any case (a unit is at most 8 values, a row at least one).
SRNL_NORM_FN int row_room(int64_t r, int64_t rows, int dim) { return rows - r > 8 ? INT_MAX : (int)(rows - r) * dim; }

// Whether the V values from column c of a row are read in one piece: its own units always, those that
// it shares with its neighbours where the kernel clips them (`clips`) and the buffer holds them whole.
// Rows may be shorter than a unit, so several at the end can share one that the buffer ends inside.
SRNL_NORM_FN bool unit_in_one_piece(int c, int V, int dim, int room, bool clips) {
  return clips ? c + V <= room : c >= 0 && c + V <= dim;
}

}  // namespace srnl
