// rglru_grid.h -- launches of very many workgroups.
//
// A dimension of a launch holds fewer than 2^32 threads (2^23 - 1 workgroups of 512), and a larger one is refused
// only when it is made, after the kernels before it have run. So workgroups are laid out in rows of kGridX, of which
// all but the largest launches have one; those of the last row behind the last workgroup leave at once.
#pragma once

#include <hip/hip_runtime.h>

namespace rglru {

constexpr unsigned kGridX = 1u << 22;  // with 512 threads each, 2^31
constexpr long long kMaxBlocks = 0x7FFFFFFF;  // their numbers stay in an int, the rows within a dimension's 65535

inline unsigned grid_x(long long blocks) { return blocks < kGridX ? static_cast<unsigned>(blocks) : kGridX; }
inline unsigned grid_rows(long long blocks) { return static_cast<unsigned>((blocks + kGridX - 1) / kGridX); }

// This workgroup's number; `row`: its place in the dimension that has the rows.
__device__ __forceinline__ int block_of(unsigned row) { return static_cast<int>(row * kGridX + blockIdx.x); }

}  // namespace rglru
