// rglru_paged.hip -- attention of one new token per sequence over a paged key-value cache (gfx950).
//
// For sequence n of len cached tokens (the new one among them), query head h on key/value head
// h / G, and the visible positions u < len with u >= len - W or u < sinks:
//   o[n][h] = sum_u softmax_u(scale <q[n][h], K[u]>) V[u],  K[u] = k_pages[table[n][u / P]][u % P].
//
// The cache is read once and everything else is small: bound by memory. A workgroup takes one
// (sequence, key/value head, up to 16 of its query heads, chunk of the visible tiles); its four
// waves take tiles of 32 keys (16 for fp32) in turn, each with its own running maximum m, sum l and
// O, joined in LDS at the end; chunks of a row are joined by paged_join. Chunks have one length
// for all rows, so that ragged batches fill the chip evenly.
//
// The query heads of a group are the columns of both contractions, so the cache's rows feed the
// matrix cores straight from global memory, with no LDS in between:
//   S^T = K Q^T: lane (c = lane % 16, g = lane / 16) loads 16 bytes of key row c: the A operand.
//   O^T += V^T P^T: S^T leaves lane (head c, group g) with keys 4g..4g+3 of each 16: already the B
//     operand if V^T takes its k index in that order. For V^T the lane loads 16 bytes of each of
//     those 8 key rows (values 8c..8c+7); operand e (value 8c + e of the 8 keys) is put together with
//     byte permutes, 4 for 8 keys. Output tile e then has O's values 8c + e. P enters as bf16 hi + lo.
//   fp32 uses the 16x16x4 fp32 instruction: the same layouts with one value a lane, no permutes.
// K of the next tile is loaded when S has used up this tile's, V after O has: one of them is
// always in flight.
//
// Positions outside the visible set get P = 0 and their V is cleared, so what lies on their part of
// a page does not matter. Page numbers outside the pool are not followed: the row becomes NaN.
//
// A cache in e4m3 (rglru_e4m3.h) takes the same way: 16 bytes are then 16 values, converted to bf16 right before
// their use. A K row's scale is an operand of that conversion; V's goes into P, in fp32. Pairs of keys of one value
// are neighbouring bytes after one permute of two rows' words, and the conversion takes pairs: 2 permutes and 4
// conversions for 8 values of a pair of rows. N128 Hq16 dh256 W2048: 113 MB in 26 us and 4.7 us of joining (bf16 48 and
// 5): 4.3 TB/s, as a tile has half the bytes of a bf16 one behind the same two dependent loads, of its page and of its rows.
// The part of attention behind a shared prefix that each sequence has for itself (rglru_prefix.hip) is the same work:
// every chunk is then left as O, m and l for the join there.
//
// N4 Hq8 Hkv2 dh128 to 131k tokens: 401 MB in 77.9 us (5.2 TB/s; a plain copy of 1 GiB 5.2); N128 Hq16 dh256
// W2048: 224 MB in 48 us and 5 us of joining, in fp32 449 MB in 94 and 5.
#include "rglru_grid.h"
#include "rglru_paged.h"

#include <algorithm>

namespace rglru {

// The paged decoding kernel (paged_rows does it).
template <typename T, typename C, int DH, bool UNI>
__global__ __launch_bounds__(64 * kPgWaves, 2) void paged_fwd(PagedArgs a, int chunk, int splits) {
  __shared__ PagedLds<DH> lds;
  paged_rows<T, C, DH, UNI, false>(a, chunk, splits, block_of(blockIdx.z), blockIdx.y, lds);
}

// Joins the chunks of the rows that have more than one: workgroup = (row, head), 4 chunk groups of
// 64 lanes with DH / 64 values each.
template <typename T, int DH>
__global__ __launch_bounds__(256) void paged_join(PagedArgs a, int chunk, int splits) {
  constexpr int V = DH / 64, kAt = 4;
  __shared__ float ro[4][DH], rl[4], rm[4];
  const int n = blockIdx.x / a.Hq, h = blockIdx.x - n * a.Hq;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int raw = uniform_load(a.lens, n);
  const size_t r0 = static_cast<size_t>(n) * splits * a.Hq + h;
  float m = a.floor, l = 0.0f, acc[V] = {};
  float2 st[kAt];
  float x[kAt][V];
  auto load = [&](int s0) {
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      const size_t r = r0 + static_cast<size_t>(min(s0 + 4 * j, splits - 1)) * a.Hq;
      st[j] = *reinterpret_cast<const float2 *>(a.stat + 2 * r);
#pragma unroll
      for (int i = 0; i < V; ++i) x[j][i] = a.part[r * DH + lane + 64 * i];
    }
  };
  // the first chunks are read before the length says how many there are (what is not used may hold
  // anything): one round trip less for the common few chunks
  load(w);
  if (raw < 0 || raw > static_cast<long long>(a.max_pages) * a.page) return;
  const Walk wk = walk_of<Paged<T, T, DH>::kKeys>(raw, a.window, a.sinks);
  if (wk.nt <= chunk) return;  // not split, or empty
  const int used = (wk.nt + chunk - 1) / chunk;
  for (int s0 = w; s0 < used; s0 += 4 * kAt) {
    if (s0 != w) load(s0);
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      if (s0 + 4 * j >= used) continue;
      const float mn = fmaxf(m, st[j].x);
      const float fo = __builtin_amdgcn_exp2f((m - mn) * a.c);
      const float fn = __builtin_amdgcn_exp2f((st[j].x - mn) * a.c);
      m = mn;
      l = fmaf(st[j].y, fn, l * fo);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(x[j][i], fn, acc[i] * fo);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) ro[w][lane + 64 * i] = acc[i];
  if (lane == 0) {
    rl[w] = l;
    rm[w] = m;
  }
  __syncthreads();
  const float mt = fmaxf(fmaxf(rm[0], rm[1]), fmaxf(rm[2], rm[3]));
  float f[4], lt = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[k] = __builtin_amdgcn_exp2f((rm[k] - mt) * a.c);
    lt = fmaf(rl[k], f[k], lt);
  }
  for (int d = threadIdx.x; d < DH; d += 256) {
    float o = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) o = fmaf(ro[k][d], f[k], o);
    Elem<T>::store(static_cast<T *>(a.o), (static_cast<size_t>(n) * a.Hq + h) * DH + d, o / lt);
  }
}

// Tiles per chunk and the most chunks a row can have. Chunks of 4 tiles (one per wave) at least;
// longer ones once all rows together give the chip enough workgroups.
PagedPlan paged_plan(int N, int Hq, int Hkv, long long max_len, int window, int sinks, int io) {
  const int keys = io == kBF16 ? 32 : 16;
  const int G = Hq / Hkv;
  const int len = static_cast<int>(std::min<long long>(max_len, 0x7FFFFF00));
  // the longest walk of any length up to len: the window's tiles may straddle one more
  const Walk w = io == kBF16 ? walk_of<32>(len, window, sinks) : walk_of<16>(len, window, sinks);
  const long long most = std::min<long long>(
      (static_cast<long long>(len) + keys - 1) / keys,
      (static_cast<long long>(std::min(window, len)) + keys - 1) / keys + 1 + w.ns);
  const long long groups = static_cast<long long>(N) * Hkv * ((G + 15) / 16);
  constexpr long long kTarget = 512;  // workgroups: two fit a CU at a time (700, 1024, 2048: slower)
  long long chunk = (most * groups + kTarget - 1) / kTarget;
  chunk = std::min(std::max<long long>(chunk, kPgWaves), most);  // (at most 2^27, as len is below 2^31)
  PagedPlan p;
  p.chunk = static_cast<int>(chunk);
  p.splits = static_cast<int>((most + chunk - 1) / chunk);
  return p;
}

namespace {

template <typename T, typename C, int DH> hipError_t launch(const PagedArgs &a, const PagedPlan &p, hipStream_t s) {
  const int G = a.Hq / a.Hkv;
  const long long cols = static_cast<long long>(a.N) * p.splits;
  const dim3 grid(grid_x(cols), a.Hkv * ((G + 15) / 16), grid_rows(cols));
  // Registers would let a third workgroup onto a CU at dh 128. That hides the latency of short walks, but on longer ones
  // three share what two can use, and of few workgroups some CUs get more than their share: LDS for two then. Hq8 Hkv2,
  // lengths spread to L, us with two and three: bf16, pages of 32: 10 tiles a workgroup N300 L300 14.7 and 14.2, N2000 69.3
  // and 62.8; 19 tiles N300 L600 21.2 and 22.1, N1000 59.8 and 58.1; 25 tiles N600 L800 43.3 and 44.6; 125 tiles N300 L4000
  // 136 and 145, N2000 723 and 729. fp32, pages of 24: 11 tiles N2000 L150 81.1 and 70.6; 20 tiles N300 L300 27.1 and 28.4,
  // N2000 137.5 and 133.5; 38 tiles N2000 L600 240 and 246; 251 tiles N300 L4000 286 and 338. (e4m3 and dh 64 lose more than
  // they win.)
  constexpr unsigned kThird = 21504;  // with the 33680 bytes of PagedLds, more than a third of 160 KB
  const bool two = DH == 128 && sizeof(C) > 1 && p.chunk >= 20;
  if (a.page % 16 == 0)
    paged_fwd<T, C, DH, true><<<grid, 64 * kPgWaves, two ? kThird : 0, s>>>(a, p.chunk, p.splits);
  else
    paged_fwd<T, C, DH, false><<<grid, 64 * kPgWaves, two ? kThird : 0, s>>>(a, p.chunk, p.splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  // (rows are split only where they are few: N * Hq is at most 16 * 512, see paged_plan)
  paged_join<T, DH><<<static_cast<unsigned>(a.N) * a.Hq, 256, 0, s>>>(a, p.chunk, p.splits);
  return hipGetLastError();
}

template <typename T, typename C> hipError_t launch(const PagedArgs &a, const PagedPlan &p, hipStream_t s) {
  switch (a.dh) {
    case 64: return launch<T, C, 64>(a, p, s);
    case 128: return launch<T, C, 128>(a, p, s);
    case 256: return launch<T, C, 256>(a, p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_paged_attention(const PagedArgs &a, const PagedPlan &p, int io, hipStream_t s) {
  if (a.k_scales) return launch<bf16_t, uint8_t>(a, p, s);
  return io == kBF16 ? launch<bf16_t, bf16_t>(a, p, s) : launch<float, float>(a, p, s);
}

}  // namespace rglru
