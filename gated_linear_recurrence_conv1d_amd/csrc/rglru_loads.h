// rglru_loads.h -- loads that the attention block's kernels share.
#pragma once

#include "rglru_mfma.h"

namespace rglru {

// dma_16b with 4 bytes per lane (256 bytes).
__device__ __forceinline__ void dma_4b(__amdgpu_buffer_rsrc_t rsrc, unsigned voff,
                                       unsigned lds_base) {
  unsigned saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %1, %3, 0 offen lds\n\t"
      "s_nop 0\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(voff), "s"(lds_base), "s"(rsrc));
}

// A value of a table that the kernel does not write, at a wave-uniform place: by scalar load.
template <typename V> __device__ __forceinline__ V uniform_load(const V *p, long long i) {
  typedef const __attribute__((address_space(4))) V *const_ptr;
  return ((const_ptr)p)[i];
}

}  // namespace rglru
