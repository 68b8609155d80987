// rglru_paged.h -- what the kernels over a paged cache share: the walk over a row's visible tiles.
#pragma once

#include "rglru_launch.h"
#include "rglru_loads.h"

namespace rglru {

// Tiles a row has to walk: first those that hold sinks before the window's first tile, then the
// window's. Host and device use the same arithmetic.
struct Walk {
  int len, w0, ns, win, nt;  // window start; sink tiles; window's first tile; tiles in all
};
template <int KEYS> __host__ __device__ inline Walk walk_of(int len, int W, int sinks) {
  Walk w;
  w.len = len;
  w.w0 = len > W ? len - W : 0;
  const int s = sinks < w.w0 ? sinks : w.w0;  // sinks beyond w0 are in the window anyway
  w.win = w.w0 / KEYS;
  w.ns = (s + KEYS - 1) / KEYS;
  if (w.ns > w.win) w.ns = w.win;
  w.nt = len > 0 ? w.ns + (len + KEYS - 1) / KEYS - w.win : 0;
  return w;
}

// The shared prefix's length, -1 if it is no length that the table can hold.
__device__ __forceinline__ int prefix_of(const int *prefix_len, long long cap) {
  const int p = uniform_load(prefix_len, 0);
  return p < 0 || p > cap ? -1 : p;
}

// How many of a row's own tokens are sinks, the prefix's tokens coming first.
__device__ __forceinline__ int sinks_behind(const PagedArgs &a) {
  const int p = prefix_of(a.prefix_len, a.prefix_cap);
  return max(0, a.sinks - max(p, 0));
}

}  // namespace rglru
