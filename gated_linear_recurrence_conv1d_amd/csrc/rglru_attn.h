// rglru_attn.h -- what the local attention kernels share: blocks of key, value or query rows in LDS, how
// they are filled and read as MFMA operands, and the mask.
//
// Rows arrive by direct buffer-to-LDS loads. The 16-byte chunk c of row r lies at c ^ f(r), with f chosen
// so that both the row reads (16 consecutive rows at one chunk) and the transposing reads (4
// consecutive rows at 4 consecutive chunks) of a pass fall on different banks.
#pragma once

#include "rglru_loads.h"
#include "rglru_shares.h"

namespace rglru {
namespace attn {

constexpr int kRawWord3 = 0x00020000;  // buffer descriptor word 3: raw 32-bit data, no swizzle
constexpr float kLn2Inv = 1.4426950408889634f;

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4_t;
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) u32x2_t lds_u32x2_t;
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// An integer that is the same in every lane, kept in a scalar register (quotients and some minima run on
// the vector unit; branches on such values, and descriptors made from them, then cost registers).
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ long long uni64(long long v) {
  const unsigned lo = __builtin_amdgcn_readfirstlane(static_cast<unsigned>(v));
  const unsigned hi = __builtin_amdgcn_readfirstlane(static_cast<unsigned>(static_cast<unsigned long long>(v) >> 32));
  return static_cast<long long>(static_cast<unsigned long long>(hi) << 32 | lo);
}

// A block of kBlk rows of DH bf16 in LDS, and the ways it is filled and read.
template <int DH, int WAVES = kWg> struct Blk {  // WAVES: how many share the loads
  static constexpr unsigned kRowBytes = DH * 2;
  static constexpr unsigned kBytes = kBlk * kRowBytes;  // one block
  static constexpr unsigned kSlot = 2 * kBytes;         // a ring slot: a block of K (Q), one of V (dO)
  static constexpr int kCPR = DH / 8;                 // 16-byte chunks per row
  static constexpr int kRPI = 64 / kCPR;              // rows per wave-wide 16-byte load
  static constexpr int kLPW = kBlk / kRPI / WAVES;    // loads per wave and block
  static constexpr int kKS = DH / 16;                 // k-steps over d
  static constexpr int kDT = DH / 32;                 // 32-wide d tiles
  // chunk swizzle: rows of 128 bytes (DH 64) share a 256-byte bank line in pairs
  __device__ __forceinline__ static int swz(int r) {
    return DH == 64 ? 4 * ((r >> 1) & 1) + ((r >> 2) & 3) : 4 * (r & 3) + ((r >> 2) & 3);
  }
  // the buffer of a block's rows: those of the sequence from `base` on, at most kBlk (rows past its
  // end then read zero, whatever lies there; rows <= 0: all)
  __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rsrc(const bf16_t *base,
                                                                unsigned row_bytes, int rows) {
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<bf16_t *>(wave_uniform(base)), static_cast<short>(0),
        rows > 0 ? static_cast<int>(row_bytes * static_cast<unsigned>(min(rows, kBlk) - 1)) + DH * 2 : 0,
        kRawWord3);
  }
  // A wave's ii-th load of a block covers rows kPart ii + (its first) ..; the lane's byte offset in it
  // depends on ii only through the chunk swizzle, whose bits repeat after kPar loads.
  static constexpr int kPart = WAVES * kRPI;
  static constexpr int kPar = kPart < 16 ? 16 / kPart : 1;
  struct Lane {
    unsigned off[kPar];
  };
  __device__ __forceinline__ static Lane load_lane(int w, int lane, unsigned row_bytes) {
    const int row = w * kRPI + lane / kCPR;
    Lane l;
#pragma unroll
    for (int p = 0; p < kPar; ++p)
      l.off[p] = static_cast<unsigned>(row) * row_bytes +
                 static_cast<unsigned>(((lane % kCPR) ^ swz(row + kPart * p)) * 16);
    return l;
  }
  // that load, from the block's buffer to its LDS byte address dst. (One buffer for all of a block's loads:
  // one for each would cost some 25 scalar instructions a load, as many cycles as the block's MFMAs at DH 128.)
  __device__ __forceinline__ static void load(__amdgpu_buffer_rsrc_t src, unsigned row_bytes, int ii, int w,
                                              const Lane &l, unsigned dst) {
    dma_16b(src, l.off[ii % kPar] + ii * kPart * row_bytes,
            static_cast<unsigned>(uni(dst + (w + WAVES * ii) * 1024)));
  }
  // A block's two reads, from byte addresses that depend on the lane only through one register: the
  // row length and every block start are multiples of the bits that the steps change by XOR.
  // row_lane / col_lane: the lane's part for step 0, to be added to the block's address.
  __device__ __forceinline__ static unsigned row_lane(int lane) {
    const int r = lane & 31;
    return r * kRowBytes + (((lane >> 5) ^ swz(r)) * 16);
  }
  // A operand, k = d of step s: 8 values of row lane % 32
  __device__ __forceinline__ static bf16x8_t rows(unsigned at, int s) {
    return __builtin_bit_cast(bf16x8_t, *(lds_u32x4_t *)static_cast<uintptr_t>(at ^ (32u * s)));
  }
  __device__ __forceinline__ static unsigned col_lane(int lane) {
    const int half = lane >> 5, r4 = (lane & 15) >> 2;
    const int cl = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int rj = DH == 64 ? r4 >> 1 : r4;
    return (4 * half + r4) * kRowBytes + 64 * rj + 16 * (cl ^ half) + 8 * (lane & 1);
  }
  // A operand, rows d = 32 j + lane % 32, k = block rows 16 st + (4 h.., 8 + 4 h..), h = lane / 32:
  // the accumulator's row order
  __device__ __forceinline__ static bf16x8_t cols(unsigned at, int st, int j) {
    const unsigned p = (at ^ (64u * j)) + 16 * st * kRowBytes;
    const i16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)static_cast<uintptr_t>(p));
    const i16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_i16x4_t *)static_cast<uintptr_t>((at ^ (64u * j) ^ 32u) + (16 * st + 8) * kRowBytes));
    const uint2 ux = __builtin_bit_cast(uint2, x), uy = __builtin_bit_cast(uint2, y);
    const u32x4_t u = {ux.x, ux.y, uy.x, uy.y};
    return __builtin_bit_cast(bf16x8_t, u);
  }
};

// A wave's 32 rows of DH bf16, one row per lane pair (l, l + 32), on their way to and from registers. Lane
// by lane, each access would touch 32 rows 16 bytes at a time; through a block of LDS that is the wave's own
// (`tile`), whole rows are read and written.
template <int DH> struct Tile {
  typedef Blk<DH, 1> K;
  static constexpr int kPasses = K::kKS;  // wave-wide 16-byte accesses of 32 rows
  // the lane's row and chunk in pass p, and their place in the tile
  __device__ __forceinline__ static int row(int p, int lane) { return p * K::kRPI + lane / K::kCPR; }
  __device__ __forceinline__ static unsigned at(unsigned tile, int p, int lane) {
    const int r = row(p, lane);
    return tile + r * K::kRowBytes + (((lane % K::kCPR) ^ K::swz(r)) * 16);
  }
  // starts the loads of the rows of the sequence from `base` on (rows >= `rows`: zero)
  __device__ __forceinline__ static void start(const bf16_t *base, unsigned row_bytes, int rows, int lane,
                                               unsigned tile) {
    asm volatile("" : "+v"(lane));  // (as in store)
    const typename K::Lane l = K::load_lane(0, lane, row_bytes);
    const __amdgpu_buffer_rsrc_t src = K::rsrc(base, row_bytes, rows);
#pragma unroll
    for (int ii = 0; ii < K::kLPW; ++ii) K::load(src, row_bytes, ii, 0, l, tile);
  }
  __device__ __forceinline__ static void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
  // this lane's row as a B operand, k-step s: its values 16 s + 8 (lane / 32) ..
  __device__ __forceinline__ static bf16x8_t operand(unsigned tile, int lane, int s) {
    return K::rows(tile + K::row_lane(lane), s);
  }
  // stores an accumulator of DH / 32 tiles (value(j, g): its elements 4 g .. 4 g + 3 of tile j, which are
  // d = 32 j + 8 g + 4 (lane / 32) .., as bf16) to the rows below `rows`
  template <typename F>
  __device__ __forceinline__ static void store(unsigned tile, int lane, F value, bf16_t *base, size_t stride,
                                               int rows) {
    asm volatile("" : "+v"(lane));  // the lane's terms are formed here: kept from the start, they take registers
    const int r = lane & 31, half = lane >> 5;
#pragma unroll
    for (int j = 0; j < K::kDT; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(lds_u32x2_t *)static_cast<uintptr_t>(tile + r * K::kRowBytes + (((4 * j + g) ^ K::swz(r)) * 16) +
                                               8 * half) = value(j, g);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      if (row(p, lane) < rows)
        *reinterpret_cast<u32x4_t *>(base + row(p, lane) * stride + 8 * (lane % K::kCPR)) =
            *(lds_u32x4_t *)static_cast<uintptr_t>(at(tile, p, lane));
  }
};

// Query row t sees key row u (t, u < len checked apart).
__device__ __forceinline__ bool sees(int t, int u, int W, int sinks) {
  return u <= t && (u > t - W || u < sinks);
}

__device__ __forceinline__ int clamp_len(const int *lens, int b, int T) {
  return uni(lens ? min(max(uniform_load(lens, b), 0), T) : T);
}

// The key blocks that query rows q0 .. q0 + rows - 1 of a sequence of len tokens need, in order: those
// with sinks before the window's first block, then the window's.
struct BlockWalk {
  int win, ns, n;  // the window's first block; sink blocks; blocks in all
  __device__ __forceinline__ BlockWalk(int q0, int rows, int len, int W, int sinks) {
    win = uni(max(0, q0 - W + 1) / kBlk);
    ns = uni(min((sinks + kBlk - 1) / kBlk, win));
    n = uni(ns + (min(len, q0 + rows) - 1) / kBlk + 1 - win);
  }
  __device__ __forceinline__ int first_row(int i) const { return (i < ns ? i : i - ns + win) * kBlk; }
};

}  // namespace attn
}  // namespace rglru
