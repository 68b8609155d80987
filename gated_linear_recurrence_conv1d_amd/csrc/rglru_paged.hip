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
// N4 Hq8 Hkv2 dh128 to 131k tokens: 401 MB in 77.6 us (5.2 TB/s, a plain copy's rate); N128 Hq16 dh256 W2048:
// 224 MB in 50 us and 5 us of joining, in fp32 449 MB in 97 and 5.
#include "rglru_grid.h"
#include "rglru_launch.h"
#include "rglru_loads.h"
#include "rglru_mfma.h"

#include <algorithm>

namespace rglru {

namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kPgWaves = 4;

template <typename T, int DH> struct Paged {
  static constexpr bool kHalf = sizeof(T) == 2;      // bf16
  static constexpr int kKeys = kHalf ? 32 : 16;      // keys per tile
  static constexpr int kSub = kKeys / 16;            // S tiles of 16 keys
  static constexpr int kDims = kHalf ? 32 : 16;      // dims a 16-byte-per-lane K load covers
  static constexpr int kKS = DH / kDims;             // K loads per 16 keys
  static constexpr int kE = kHalf ? (DH / 16 < 8 ? DH / 16 : 8) : 4;  // values per V load and lane
  static constexpr int kVB = DH / (16 * kE);         // V loads per key row
  static constexpr int kVK = 4 * kSub;               // key rows of V per lane
  static constexpr int kVW = kE * static_cast<int>(sizeof(T)) / 4;  // 32-bit words per V load
  static constexpr int kOT = DH / 16;                // O^T tiles
  static constexpr int kLdO = DH + 1;                // LDS row of O (one word against conflicts)
  // q from LDS, tile by tile, where registers do not hold it beside K, V and O: what is spilled is read back behind the
  // loads in flight (N128 Hq16 dh256 W2048: 65 us with 9 spilled registers)
  static constexpr bool kQLds = DH == 256;
};

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

}  // namespace

// UNI: the page size is a multiple of 16, so that 16 aligned keys lie on one page: their rows' address
// is wave-uniform (one scalar table load) plus a constant offset per lane.
template <typename T, int DH, bool UNI>
__global__ __launch_bounds__(64 * kPgWaves, 2) void paged_fwd(PagedArgs a, int chunk, int splits) {
  typedef Paged<T, DH> M;
  __shared__ __attribute__((aligned(16))) float so[kPgWaves][16][M::kLdO];
  __shared__ float sm[kPgWaves][16], sl[kPgWaves][16];
  __shared__ int sbad[kPgWaves];
  u32x4_t(*const sq)[64] = reinterpret_cast<u32x4_t(*)[64]>(so);  // q lies there until the waves are joined
  static_assert(!M::kQLds || M::kKS * 64 * sizeof(u32x4_t) <= sizeof(so), "room for q");
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  const int id = block_of(blockIdx.z), n = id / splits, sp = id - n * splits;
  if (n >= a.N) return;
  const int G = a.Hq / a.Hkv, gt = (G + 15) / 16;
  const int kvh = blockIdx.y / gt;
  const int h0 = (blockIdx.y - kvh * gt) * 16;  // first head of the group's part
  const int nh = min(16, G - h0);
  const int hq = kvh * G + h0;                  // first query head
  const int raw = uniform_load(a.lens, n);
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  const bool bad_len = raw < 0 || raw > cap;
  const Walk wk = walk_of<M::kKeys>(bad_len ? 0 : raw, a.window, a.sinks);
  const int t_end = min(wk.nt, (sp + 1) * chunk);
  if (sp > 0 && sp * chunk >= wk.nt) return;    // no such chunk (chunk 0 also serves empty rows)
  const int *table = a.table + static_cast<size_t>(n) * a.max_pages;
  const size_t row_bytes = static_cast<size_t>(a.Hkv) * DH * sizeof(T);
  const char *kp = static_cast<const char *>(a.k_pages) + static_cast<size_t>(kvh) * DH * sizeof(T);
  const char *vp = static_cast<const char *>(a.v_pages) + static_cast<size_t>(kvh) * DH * sizeof(T);

  // Q^T operand: head column c16 (heads past the group read the last one; never stored)
  u32x4_t qf[M::kQLds ? 1 : M::kKS];
  {
    const T *qp = static_cast<const T *>(a.q) + static_cast<size_t>(n) * a.q_stride +
                  static_cast<size_t>(hq + min(c16, nh - 1)) * DH + g * (M::kDims / 4);
    if constexpr (M::kQLds) {
#pragma unroll
      for (int s = 0; s < M::kKS / kPgWaves; ++s) {
        const int ws = w + kPgWaves * s;
        sq[ws][lane] = *reinterpret_cast<const u32x4_t *>(qp + ws * M::kDims);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int s = 0; s < M::kKS; ++s) qf[s] = *reinterpret_cast<const u32x4_t *>(qp + s * M::kDims);
    }
  }
  f32x4_t oacc[M::kOT];
#pragma unroll
  for (int i = 0; i < M::kOT; ++i) oacc[i] = f32x4_t{};
  float m_run = a.floor, l_run = 0.0f;
  int bad = bad_len;

  auto tile_base = [&](int i) { return (i < wk.ns ? i : i - wk.ns + wk.win) * M::kKeys; };
  auto seen = [&](int u) { return u < wk.len && (u >= wk.w0 || u < a.sinks); };

  // Where tile i's rows are: UNI the first row of each 16 keys (wave-uniform), else a row per key.
  struct At {
    size_t base[M::kSub];      // UNI: byte offset of the 16 keys' first row
    int krow[M::kSub];         // else: pool rows of this lane's K keys and V keys
    int vrow[M::kVK];
  };
  auto locate = [&](int i) {
    At at;
    const int u0 = tile_base(i);
    if constexpr (UNI) {
#pragma unroll
      for (int s = 0; s < M::kSub; ++s) {
        const int u = u0 + 16 * s;
        // some of the 16 visible? (if not, their page need not be there: row 0 stands in)
        const bool need = u < wk.len && (u + 16 > wk.w0 || u < a.sinks);
        int page = 0, first = 0;
        if (need) {
          const int t = u / a.page;
          page = uniform_load(table, t);
          first = u - t * a.page;
          if (page < 0 || page >= a.num_pages) {
            bad = 1;
            page = first = 0;
          }
        }
        at.base[s] = (static_cast<size_t>(page) * a.page + first) * row_bytes;
      }
    } else {
      const int u = u0 + (lane & (M::kKeys - 1));
      int row = 0;
      if (seen(u)) {
        const int t = u / a.page, p = table[t];
        if (p < 0 || p >= a.num_pages)
          bad = 1;
        else
          row = p * a.page + (u - t * a.page);
      }
#pragma unroll
      for (int s = 0; s < M::kSub; ++s) at.krow[s] = __shfl(row, 16 * s + c16, 64);
#pragma unroll
      for (int k = 0; k < M::kVK; ++k) at.vrow[k] = __shfl(row, 16 * (k >> 2) + 4 * g + (k & 3), 64);
    }
    return at;
  };
  u32x4_t kf[M::kSub][M::kKS];
  uint32_t vf[M::kVK][M::kVB][M::kVW];
  const unsigned kof = static_cast<unsigned>(c16 * row_bytes) + g * 16;
  const unsigned vof = static_cast<unsigned>(4 * g * row_bytes) + c16 * (M::kE * sizeof(T));
  auto load_k = [&](const At &at) {
#pragma unroll
    for (int s = 0; s < M::kSub; ++s) {
      const char *p;
      if constexpr (UNI)
        p = wave_uniform(kp + at.base[s]) + kof;
      else
        p = kp + static_cast<size_t>(at.krow[s]) * row_bytes + g * 16;
#pragma unroll
      for (int i = 0; i < M::kKS; ++i) kf[s][i] = *reinterpret_cast<const u32x4_t *>(p + i * 64);
    }
  };
  auto load_v = [&](const At &at) {
#pragma unroll
    for (int k = 0; k < M::kVK; ++k) {
      const char *p;
      if constexpr (UNI)
        p = wave_uniform(vp + at.base[k >> 2] + (k & 3) * row_bytes) + vof;
      else
        p = vp + static_cast<size_t>(at.vrow[k]) * row_bytes + c16 * (M::kE * sizeof(T));
#pragma unroll
      for (int b = 0; b < M::kVB; ++b) {
        const char *pb = p + b * 16 * M::kE * sizeof(T);
        if constexpr (M::kVW == 4) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t *>(pb);
#pragma unroll
          for (int e = 0; e < 4; ++e) vf[k][b][e] = v[e];
        } else {
          const u32x2_t v = *reinterpret_cast<const u32x2_t *>(pb);
          vf[k][b][0] = v[0];
          vf[k][b][1] = v[1];
        }
      }
    }
  };

  const int t0 = sp * chunk + w;
  if (t0 < t_end) {
    At at = locate(t0);
    load_k(at);
    load_v(at);
    if (t0 + kPgWaves < t_end) at = locate(t0 + kPgWaves);
    for (int i = t0; i < t_end; i += kPgWaves) {
      const bool more = i + kPgWaves < t_end;
      const int u0 = tile_base(i);
      // ---- S^T of the tile
      f32x4_t s[M::kSub];
#pragma unroll
      for (int j = 0; j < M::kSub; ++j) s[j] = f32x4_t{};
      int ql = lane;
      asm volatile("" : "+v"(ql));  // read in every tile: kept, q would take registers again
#pragma unroll
      for (int d = 0; d < M::kKS; ++d) {
        const u32x4_t qd = M::kQLds ? sq[d][ql] : qf[M::kQLds ? 0 : d];
#pragma unroll
        for (int j = 0; j < M::kSub; ++j) {
          if constexpr (M::kHalf) {
            s[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, kf[j][d]),
                                                           __builtin_bit_cast(bf16x8_t, qd), s[j], 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kf[j][d][e]),
                                                          __uint_as_float(qd[e]), s[j], 0, 0, 0);
          }
        }
      }
      if (more) load_k(at);
      // ---- mask: tiles that are not visible throughout
      const bool full = u0 + M::kKeys <= wk.len && (u0 >= wk.w0 || u0 + M::kKeys <= a.sinks);
      if (!full) {
#pragma unroll
        for (int k = 0; k < M::kVK; ++k) {
          const bool on = seen(u0 + 16 * (k >> 2) + 4 * g + (k & 3));
          s[k >> 2][k & 3] = on ? s[k >> 2][k & 3] : -__builtin_inff();
#pragma unroll
          for (int b = 0; b < M::kVB; ++b)
#pragma unroll
            for (int e = 0; e < M::kVW; ++e) vf[k][b][e] = on ? vf[k][b][e] : 0u;
        }
      }
      // ---- running softmax; the maximum is raised only when it grows by more than 2^8 (O and l
      // share it, so the result does not change)
      float mx = a.floor;
#pragma unroll
      for (int k = 0; k < M::kVK; ++k) mx = fmaxf(mx, s[k >> 2][k & 3]);
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const bool raise = (mx - m_run) * a.c > 8.0f;
      if (__any(raise)) {
        const float m_new = raise ? mx : m_run;
        const float corr = __builtin_amdgcn_exp2f((m_run - m_new) * a.c);
        l_run *= corr;
        m_run = m_new;
#pragma unroll
        for (int t = 0; t < M::kOT; ++t) oacc[t] *= corr;
      }
      float p[M::kVK];
#pragma unroll
      for (int k = 0; k < M::kVK; ++k) {
        p[k] = __builtin_amdgcn_exp2f((s[k >> 2][k & 3] - m_run) * a.c);
        l_run += p[k];
      }
      // ---- O^T += V^T P^T
      if constexpr (M::kHalf) {
        // P as bf16 hi + lo: bf16 alone would be most of o's error, and the second product is hardly seen beside the
        // cache's bytes (N4 to 131k tokens 77.0 -> 77.6 us, N1 11.5 -> 11.7; N128 56.4 -> 55.7 with q in LDS)
        u32x4_t ph, pl;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ph[k] = pack_bf16x2(p[2 * k], p[2 * k + 1]);
          pl[k] = pack_bf16x2(p[2 * k] - bf16lo(ph[k]), p[2 * k + 1] - bf16hi(ph[k]));
        }
#pragma unroll
        for (int b = 0; b < M::kVB; ++b)
#pragma unroll
          for (int e = 0; e < M::kE; ++e) {
            u32x4_t v;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] = __builtin_amdgcn_perm(vf[2 * k + 1][b][e / 2], vf[2 * k][b][e / 2],
                                           e & 1 ? 0x07060302u : 0x05040100u);
            f32x4_t &o = oacc[b * M::kE + e];
            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v),
                                                        __builtin_bit_cast(bf16x8_t, ph), o, 0, 0, 0);
            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v),
                                                        __builtin_bit_cast(bf16x8_t, pl), o, 0, 0, 0);
          }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int b = 0; b < M::kVB; ++b)
#pragma unroll
            for (int e = 0; e < M::kE; ++e)
              oacc[b * M::kE + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  __uint_as_float(vf[k][b][e]), p[k], oacc[b * M::kE + e], 0, 0, 0);
      }
      if (more) {
        load_v(at);
        if (i + 2 * kPgWaves < t_end) at = locate(i + 2 * kPgWaves);
      }
    }
  }
  // ---- join the four waves
  l_run += __shfl_xor(l_run, 16, 64);
  l_run += __shfl_xor(l_run, 32, 64);
  const bool any_bad = __any(bad);
  if (g == 0) {
    sm[w][c16] = m_run;
    sl[w][c16] = l_run;
  }
  if (lane == 0) sbad[w] = any_bad;
  __syncthreads();
  float M4 = sm[0][c16];
#pragma unroll
  for (int i = 1; i < kPgWaves; ++i) M4 = fmaxf(M4, sm[i][c16]);
  const float f = __builtin_amdgcn_exp2f((m_run - M4) * a.c);
  // a wave's weight is 0 where it saw nothing, and its O is 0 then
#pragma unroll
  for (int t = 0; t < M::kOT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = (t / M::kE) * 16 * M::kE + (4 * g + j) * M::kE + t % M::kE;
      if (c16 < nh) so[w][c16][d] = oacc[t][j] * f;
    }
  __syncthreads();
  const bool isbad = sbad[0] | sbad[1] | sbad[2] | sbad[3];
  const bool partial = wk.nt > chunk;  // the row has other chunks
  for (int i = threadIdx.x; i < nh * DH; i += 64 * kPgWaves) {
    const int h = i / DH, d = i - h * DH;
    float Mh = sm[0][h];
#pragma unroll
    for (int k = 1; k < kPgWaves; ++k) Mh = fmaxf(Mh, sm[k][h]);
    float l = 0.0f, o = 0.0f;
#pragma unroll
    for (int k = 0; k < kPgWaves; ++k) {
      l = fmaf(sl[k][h], __builtin_amdgcn_exp2f((sm[k][h] - Mh) * a.c), l);
      o += so[k][h][d];
    }
    if (isbad) l = __builtin_nanf("");
    if (partial) {
      const size_t r = (static_cast<size_t>(n) * splits + sp) * a.Hq + hq + h;
      a.part[r * DH + d] = o;
      if (d == 0) {
        a.stat[2 * r] = Mh;
        a.stat[2 * r + 1] = l;
      }
    } else {
      const float r = isbad ? l : wk.nt == 0 ? 0.0f : o / l;
      Elem<T>::store(static_cast<T *>(a.o), (static_cast<size_t>(n) * a.Hq + hq + h) * DH + d, r);
    }
  }
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
  const Walk wk = walk_of<Paged<T, DH>::kKeys>(raw, a.window, a.sinks);
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
  chunk = std::max<long long>(chunk, kPgWaves);
  PagedPlan p;
  p.chunk = static_cast<int>(std::min<long long>(chunk, 1 << 28));
  p.splits = static_cast<int>((most + p.chunk - 1) / p.chunk);
  if (p.splits < 1) p.splits = 1;
  return p;
}

namespace {

template <typename T, int DH> hipError_t launch(const PagedArgs &a, const PagedPlan &p, hipStream_t s) {
  const int G = a.Hq / a.Hkv;
  const long long cols = static_cast<long long>(a.N) * p.splits;
  const dim3 grid(grid_x(cols), a.Hkv * ((G + 15) / 16), grid_rows(cols));
  if (a.page % 16 == 0)
    paged_fwd<T, DH, true><<<grid, 64 * kPgWaves, 0, s>>>(a, p.chunk, p.splits);
  else
    paged_fwd<T, DH, false><<<grid, 64 * kPgWaves, 0, s>>>(a, p.chunk, p.splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  // (rows are split only where they are few: N * Hq is at most 16 * 512, see paged_plan)
  paged_join<T, DH><<<static_cast<unsigned>(a.N) * a.Hq, 256, 0, s>>>(a, p.chunk, p.splits);
  return hipGetLastError();
}

template <typename T> hipError_t launch(const PagedArgs &a, const PagedPlan &p, hipStream_t s) {
  switch (a.dh) {
    case 64: return launch<T, 64>(a, p, s);
    case 128: return launch<T, 128>(a, p, s);
    case 256: return launch<T, 256>(a, p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_paged_attention(const PagedArgs &a, const PagedPlan &p, int io, hipStream_t s) {
  return io == kBF16 ? launch<bf16_t>(a, p, s) : launch<float>(a, p, s);
}

}  // namespace rglru
