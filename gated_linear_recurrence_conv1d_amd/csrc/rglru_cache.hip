// rglru_cache.hip -- a paged key-value cache in e4m3: rows quantised as they are written, and read back (gfx950).
//
//   write: for row r, head h of k and of v: s = scale of the dh values (rglru_e4m3.h), codes = e4m3(x / s), both to
//          cache row slots[r];   read: out[b][t][h] = codes * s of token starts[b] + t of sequence b.
//
// Both are bound by memory and touch each byte once. A thread has 8 values of k and the same 8 of v: 16-byte accesses
// on the bf16 side, 8-byte ones on the codes' side, both runs without holes over the heads of a row. The 8 .. 32 lanes
// of a head find its largest magnitude by lane exchanges; as integers, so that a NaN wins.
//
// 16384 fp32 rows of Hkv2 dh128: written in 8.4 us (42 MB, 5.0 TB/s), 65000 read back in 30 us (166 MB, 5.5 TB/s; a
// plain copy of 256 MB reaches 5.4); 8 times 2048 bf16 rows of dh256 read back in 6.5 us (25 MB).
#include "rglru_e4m3.h"
#include "rglru_grid.h"
#include "rglru_launch.h"
#include "rglru_loads.h"

namespace rglru {

namespace {

constexpr int kPer = 8;         // values per thread
constexpr int kThreadsC = 256;  // per workgroup

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

template <typename T> struct Eight {
  float x[kPer];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (sizeof(T) == 2) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t *>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo(v[i]);
        x[2 * i + 1] = bf16hi(v[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32x4_t v = reinterpret_cast<const u32x4_t *>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = __uint_as_float(v[j]);
      }
    }
  }
};

// 8 codes times s
template <typename T> __device__ __forceinline__ void store_eight(T *p, u32x2_t codes, float s) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[2 * i] = bf16x2_of<false>(codes[i], s);
    v[2 * i + 1] = bf16x2_of<true>(codes[i], s);
  }
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<u32x4_t *>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4_t f = {v[2 * i] << 16, v[2 * i] & 0xffff0000u, v[2 * i + 1] << 16, v[2 * i + 1] & 0xffff0000u};
      reinterpret_cast<u32x4_t *>(p)[i] = f;
    }
  }
}

// Largest of N neighbouring lanes' values (N a power of two), in every one of them.
template <int N> __device__ __forceinline__ unsigned group_max(unsigned v) {
#pragma unroll
  for (int o = 1; o < N; o <<= 1) v = max(v, static_cast<unsigned>(__shfl_xor(static_cast<int>(v), o, 64)));
  return v;
}

}  // namespace

template <typename T, int DH>
__global__ __launch_bounds__(kThreadsC) void cache_quantize(CacheWriteArgs a) {
  constexpr int LPH = DH / kPer;  // lanes per head
  const long long i = static_cast<long long>(block_of(blockIdx.y)) * kThreadsC + threadIdx.x;
  const int per_row = a.Hkv * LPH;
  const long long row = i / per_row;
  if (row >= a.rows) return;
  const int c = static_cast<int>(i - row * per_row);  // which 8 values of the row
  const long long slot = a.slots[row];
  if (slot < 0 || slot >= a.n_slots) return;  // (a row's lanes leave together: the exchanges stay within a head)
  Eight<T> e[2];
  e[0].load(static_cast<const T *>(a.k) + row * a.k_stride + c * kPer);
  e[1].load(static_cast<const T *>(a.v) + row * a.v_stride + c * kPer);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float(&x)[kPer] = e[w].x;
    unsigned top = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    const unsigned b = scale_of(group_max<LPH>(top));
    u32x2_t codes = {0x7F7F7F7Fu, 0x7F7F7F7Fu};  // NaN
    if (b != kScaleNan) {
      const float r = inverse_scale(b);
#pragma unroll
      for (int j = 0; j < 2; ++j) codes[j] = pack_e4m3(x[4 * j] * r, x[4 * j + 1] * r, x[4 * j + 2] * r, x[4 * j + 3] * r);
    }
    uint8_t *const pages = static_cast<uint8_t *>(w ? a.v_pages : a.k_pages);
    uint8_t *const scales = static_cast<uint8_t *>(w ? a.v_scales : a.k_scales);
    *reinterpret_cast<u32x2_t *>(pages + (slot * per_row + c) * kPer) = codes;
    if (c % LPH == 0) scales[slot * a.Hkv + c / LPH] = static_cast<uint8_t>(b);
  }
}

template <typename T, int DH>
__global__ __launch_bounds__(kThreadsC) void cache_dequantize(CacheReadArgs a, int blocks) {
  constexpr int LPH = DH / kPer;
  const int id = block_of(blockIdx.y), b = id / blocks;
  if (b >= a.B) return;
  const int per_row = a.Hkv * LPH;
  const long long i = static_cast<long long>(id - b * blocks) * kThreadsC + threadIdx.x;
  const int t = static_cast<int>(i / per_row);
  if (t >= a.T) return;
  const int c = static_cast<int>(i - static_cast<long long>(t) * per_row);
  const long long len = uniform_load(a.lens, b), start = a.starts ? uniform_load(a.starts, b) : 0;
  const size_t row = static_cast<size_t>(b) * a.T + t;
  T *const ko = static_cast<T *>(a.k_out) + row * a.k_stride + c * kPer;
  T *const vo = static_cast<T *>(a.v_out) + row * a.v_stride + c * kPer;
  u32x2_t ck = {}, cv = {};
  float sk = 1.0f, sv = 1.0f;
  bool ok = len >= 0 && len <= static_cast<long long>(a.max_pages) * a.page && start >= 0;
  if (ok) {
    const long long u = start + t;
    if (u >= len) {  // behind the sequence
      if (!a.zero_rest) return;
    } else {
      const int p = static_cast<int>(u) / a.page;
      const int page = a.table[static_cast<size_t>(b) * a.max_pages + p];
      ok = page >= 0 && page < a.num_pages;
      if (ok) {
        const size_t at = static_cast<size_t>(page) * a.page + (static_cast<int>(u) - p * a.page);
        ck = *reinterpret_cast<const u32x2_t *>(static_cast<const uint8_t *>(a.k_pages) + (at * per_row + c) * kPer);
        cv = *reinterpret_cast<const u32x2_t *>(static_cast<const uint8_t *>(a.v_pages) + (at * per_row + c) * kPer);
        const size_t h = at * a.Hkv + c / LPH;
        sk = scale_value(static_cast<const uint8_t *>(a.k_scales)[h]);
        sv = scale_value(static_cast<const uint8_t *>(a.v_scales)[h]);
      }
    }
  }
  if (!ok) ck = cv = u32x2_t{0x7F7F7F7Fu, 0x7F7F7F7Fu};
  store_eight<T>(ko, ck, sk);
  store_eight<T>(vo, cv, sv);
}

namespace {

template <typename T, int DH> hipError_t write(const CacheWriteArgs &a, hipStream_t s) {
  const long long blocks = (static_cast<long long>(a.rows) * a.Hkv * (DH / kPer) + kThreadsC - 1) / kThreadsC;
  cache_quantize<T, DH><<<dim3(grid_x(blocks), grid_rows(blocks)), kThreadsC, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int DH> hipError_t read(const CacheReadArgs &a, hipStream_t s) {
  const long long blocks = cache_read_blocks(a.T, a.Hkv, DH), all = blocks * a.B;
  cache_dequantize<T, DH><<<dim3(grid_x(all), grid_rows(all)), kThreadsC, 0, s>>>(a, static_cast<int>(blocks));
  return hipGetLastError();
}

template <typename T> hipError_t write(const CacheWriteArgs &a, int dh, hipStream_t s) {
  return dh == 64 ? write<T, 64>(a, s) : dh == 128 ? write<T, 128>(a, s) : write<T, 256>(a, s);
}

template <typename T> hipError_t read(const CacheReadArgs &a, int dh, hipStream_t s) {
  return dh == 64 ? read<T, 64>(a, s) : dh == 128 ? read<T, 128>(a, s) : read<T, 256>(a, s);
}

}  // namespace

long long cache_read_blocks(int T, int Hkv, int dh) {
  return (static_cast<long long>(T) * Hkv * (dh / kPer) + kThreadsC - 1) / kThreadsC;
}

hipError_t launch_cache_quantize(const CacheWriteArgs &a, int dh, int io, hipStream_t s) {
  return io == kBF16 ? write<bf16_t>(a, dh, s) : write<float>(a, dh, s);
}

hipError_t launch_cache_dequantize(const CacheReadArgs &a, int dh, int io, hipStream_t s) {
  return io == kBF16 ? read<bf16_t>(a, dh, s) : read<float>(a, dh, s);
}

}  // namespace rglru
