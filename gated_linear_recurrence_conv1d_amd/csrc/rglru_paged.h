// rglru_paged.h -- what the kernels over a paged cache share: the walk over a row's visible tiles, and attention over
// them (rglru_paged.hip has its description).
#pragma once

#include "rglru_e4m3.h"
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

// A load from device memory, said to the compiler: an address put together from scalar registers it takes for one that
// may be in LDS as well, and waits for both.
template <typename V> __device__ __forceinline__ V global_load(const void *p) {
  typedef const __attribute__((address_space(1))) V *global_ptr;
  return *(global_ptr)p;
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

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kPgWaves = 4;

// q and o of type T, the cache of type C: T, or uint8_t for e4m3 (T bf16).
template <typename T, typename C, int DH> struct Paged {
  static constexpr bool kCode = sizeof(C) == 1;
  static constexpr bool kHalf = sizeof(T) == 2;      // bf16
  static constexpr int kKeys = kHalf ? 32 : 16;      // keys per tile
  static constexpr int kSub = kKeys / 16;            // S tiles of 16 keys
  static constexpr int kDims = kCode ? 64 : kHalf ? 32 : 16;  // dims a 16-byte-per-lane K load covers
  static constexpr int kKS = DH / kDims;             // K loads per 16 keys
  static constexpr int kQN = kCode ? 2 * kKS : kKS;  // q operands
  static constexpr int kMost = 16 / static_cast<int>(sizeof(C));              // values of 16 bytes
  static constexpr int kE = DH / 16 < kMost ? DH / 16 : kMost;                // values per V load and lane
  static constexpr int kVB = DH / (16 * kE);         // V loads per key row
  static constexpr int kVK = 4 * kSub;               // key rows of V per lane
  static constexpr int kVW = kE * static_cast<int>(sizeof(C)) / 4;  // 32-bit words per V load
  static constexpr int kOT = DH / 16;                // O^T tiles
  // q from LDS, tile by tile, where registers do not hold it beside K, V and O: what is spilled is read back behind the
  // loads in flight (N128 Hq16 dh256 W2048: 65 us with 9 spilled registers)
  static constexpr bool kQLds = DH == 256 && !kCode;
};

// Where a workgroup's waves meet (rows of O one word longer, against conflicts).
template <int DH> struct PagedLds {
  __attribute__((aligned(16))) float o[kPgWaves][16][DH + 1];
  float m[kPgWaves][16], l[kPgWaves][16];
  int bad[kPgWaves];
  float sum[16], top[16];
};

// UNI: the page size is a multiple of 16, so that 16 aligned keys lie on one page: their rows' address
// is wave-uniform (one scalar table load) plus a constant offset per lane.
// PRE: the rows' own part behind a shared prefix.
// id, by: the workgroup's (row, chunk) and (key/value head, 16 of its query heads).
template <typename T, typename C, int DH, bool UNI, bool PRE>
__device__ __forceinline__ void paged_rows(const PagedArgs &a, int chunk, int splits, int id, int by, PagedLds<DH> &lds) {
  typedef Paged<T, C, DH> M;
  auto &so = lds.o;
  auto &sm = lds.m;
  auto &sl = lds.l;
  auto &sbad = lds.bad;
  u32x4_t(*const sq)[64] = reinterpret_cast<u32x4_t(*)[64]>(so);  // q lies there until the waves are joined
  static_assert(!M::kQLds || M::kQN * 64 * sizeof(u32x4_t) <= sizeof(so), "room for q");
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  const int n = id / splits, sp = id - n * splits;
  if (n >= a.N) return;
  const int G = a.Hq / a.Hkv, gt = (G + 15) / 16;
  const int kvh = by / gt;
  const int h0 = (by - kvh * gt) * 16;  // first head of the group's part
  const int nh = min(16, G - h0);
  const int hq = kvh * G + h0;                  // first query head
  const int raw = uniform_load(a.lens, n);
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  const bool bad_len = raw < 0 || raw > cap;
  const int sinks = PRE ? sinks_behind(a) : a.sinks;
  const Walk wk = walk_of<M::kKeys>(bad_len ? 0 : raw, a.window, sinks);
  if (PRE && wk.nt == 0) return;                // the join knows
  const int t_end = min(wk.nt, (sp + 1) * chunk);
  if (sp > 0 && sp * chunk >= wk.nt) return;    // no such chunk (chunk 0 also serves empty rows)
  const int *table = a.table + static_cast<size_t>(n) * a.max_pages;
  const size_t row_bytes = static_cast<size_t>(a.Hkv) * DH * sizeof(C);
  const char *kp = static_cast<const char *>(a.k_pages) + static_cast<size_t>(kvh) * DH * sizeof(C);
  const char *vp = static_cast<const char *>(a.v_pages) + static_cast<size_t>(kvh) * DH * sizeof(C);

  // Q^T operand: head column c16 (heads past the group read the last one; never stored)
  u32x4_t qf[M::kQLds ? 1 : M::kQN];
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
      for (int s = 0; s < M::kQN; ++s)
        qf[s] = *reinterpret_cast<const u32x4_t *>(qp + (M::kCode ? (s >> 1) * M::kDims + (s & 1) * 8 : s * M::kDims));
    }
  }
  f32x4_t oacc[M::kOT];
#pragma unroll
  for (int i = 0; i < M::kOT; ++i) oacc[i] = f32x4_t{};
  float m_run = a.floor, l_run = 0.0f;
  int bad = bad_len;

  auto tile_base = [&](int i) { return (i < wk.ns ? i : i - wk.ns + wk.win) * M::kKeys; };
  auto seen = [&](int u) { return u < wk.len && (u >= wk.w0 || u < sinks); };

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
        const bool need = u < wk.len && (u + 16 > wk.w0 || u < sinks);
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
  const unsigned vof = static_cast<unsigned>(4 * g * row_bytes) + c16 * (M::kE * sizeof(C));
  // e4m3: the scales of this lane's K rows, and V's of key lane % 32 of the tile
  unsigned ksc[M::kCode ? M::kSub : 1], vsc = 0;
  auto scale_at = [&](const At &at, int s) {  // key c16 of the s-th 16 keys
    if constexpr (UNI)
      return at.base[s] / DH + static_cast<size_t>(c16) * a.Hkv + kvh;  // (row_bytes / DH is Hkv)
    else
      return static_cast<size_t>(at.krow[s]) * a.Hkv + kvh;
  };
  // The address of a row's loads stays until all of them are on their way: a load whose result goes over it would not
  // follow the one before it at once (fp32, pages of 24, dh 128, N64 Hq8 Hkv2 to 4000 tokens: 66.6 -> 63.5 us; pages of 32
  // 61.0 -> 59.5; where a row is one or two loads by addresses of each lane's own, dh 64, it costs 2%).
  auto keep = [&](const char *p) {
    if constexpr (DH > 64 || UNI) asm volatile("" ::"v"(p));
  };
  auto load_k = [&](const At &at) {
    if constexpr (M::kCode)
#pragma unroll
      for (int s = 0; s < M::kSub; ++s) ksc[s] = static_cast<const uint8_t *>(a.k_scales)[scale_at(at, s)];
#pragma unroll
    for (int s = 0; s < M::kSub; ++s) {
      const char *p;
      if constexpr (UNI)
        p = wave_uniform(kp + at.base[s]) + kof;
      else
        p = kp + static_cast<size_t>(at.krow[s]) * row_bytes + g * 16;
#pragma unroll
      for (int i = 0; i < M::kKS; ++i) kf[s][i] = global_load<u32x4_t>(p + i * 64);
      keep(p);
    }
  };
  auto load_v = [&](const At &at) {
    if constexpr (M::kCode)
      vsc = static_cast<const uint8_t *>(a.v_scales)[lane & 16 ? scale_at(at, M::kSub - 1) : scale_at(at, 0)];
#pragma unroll
    for (int k = 0; k < M::kVK; ++k) {
      const char *p;
      if constexpr (UNI)
        p = wave_uniform(vp + at.base[k >> 2] + (k & 3) * row_bytes) + vof;
      else
        p = vp + static_cast<size_t>(at.vrow[k]) * row_bytes + c16 * (M::kE * sizeof(C));
#pragma unroll
      for (int b = 0; b < M::kVB; ++b) {
        const char *pb = p + b * 16 * M::kE * sizeof(C);
        if constexpr (M::kVW == 4) {
          const u32x4_t v = global_load<u32x4_t>(pb);
#pragma unroll
          for (int e = 0; e < 4; ++e) vf[k][b][e] = v[e];
        } else if constexpr (M::kVW == 2) {
          const u32x2_t v = global_load<u32x2_t>(pb);
          vf[k][b][0] = v[0];
          vf[k][b][1] = v[1];
        } else {
          vf[k][b][0] = global_load<uint32_t>(pb);
        }
      }
      keep(p);
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
      for (int d = 0; d < M::kQN; ++d) {
        const u32x4_t qd = M::kQLds ? sq[d][ql] : qf[M::kQLds ? 0 : d];
#pragma unroll
        for (int j = 0; j < M::kSub; ++j) {
          if constexpr (M::kCode) {
            const float sc = __uint_as_float(ksc[M::kCode ? j : 0] << 23);  // (the exponent's field)
            u32x4_t k8;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t codes = kf[j][d >> 1][2 * (d & 1) + (e >> 1)];
              k8[e] = e & 1 ? bf16x2_of<true>(codes, sc) : bf16x2_of<false>(codes, sc);
            }
            s[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, k8),
                                                           __builtin_bit_cast(bf16x8_t, qd), s[j], 0, 0, 0);
          } else if constexpr (M::kHalf) {
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
      const bool full = u0 + M::kKeys <= wk.len && (u0 >= wk.w0 || u0 + M::kKeys <= sinks);
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
      if constexpr (M::kCode) {
        const float vs = scale_value(vsc);
#pragma unroll
        for (int k = 0; k < M::kVK; ++k) {
          const float f = __shfl(vs, 16 * (k >> 2) + 4 * g + (k & 3), 64);
          p[k] = full || seen(u0 + 16 * (k >> 2) + 4 * g + (k & 3)) ? p[k] * f : 0.0f;  // (f may be NaN where unseen)
        }
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
            if constexpr (M::kCode) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                // values e and e ^ 1 of the two rows, as (row, row + 1) pairs
                const uint32_t two = __builtin_amdgcn_perm(vf[2 * k + 1][b][e / 4], vf[2 * k][b][e / 4],
                                                           e & 2 ? 0x07030602u : 0x05010400u);
                v[k] = e & 1 ? bf16x2_of<true>(two, 1.0f) : bf16x2_of<false>(two, 1.0f);
              }
            } else
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
  if (w == 0 && g == 0) {  // the head's sum over the waves
    float l = 0.0f;
#pragma unroll
    for (int k = 0; k < kPgWaves; ++k) l = fmaf(sl[k][c16], __builtin_amdgcn_exp2f((sm[k][c16] - M4) * a.c), l);
    lds.sum[c16] = sbad[0] | sbad[1] | sbad[2] | sbad[3] ? __builtin_nanf("") : l;
    lds.top[c16] = M4;
  }
  // a wave's weight is 0 where it saw nothing, and its O is 0 then
#pragma unroll
  for (int t = 0; t < M::kOT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = (t / M::kE) * 16 * M::kE + (4 * g + j) * M::kE + t % M::kE;
      if (c16 < nh) so[w][c16][d] = oacc[t][j] * f;
    }
  __syncthreads();
  const bool partial = PRE || wk.nt > chunk;  // the row has other chunks
  for (int i = threadIdx.x; i < nh * DH; i += 64 * kPgWaves) {
    const int h = i / DH, d = i - h * DH;
    const float l = lds.sum[h];
    float o = 0.0f;
#pragma unroll
    for (int k = 0; k < kPgWaves; ++k) o += so[k][h][d];
    if (partial) {
      const size_t r = (static_cast<size_t>(n) * (PRE ? a.parts : splits) + (PRE ? a.first_part : 0) + sp) * a.Hq + hq + h;
      a.part[r * DH + d] = o;
      if (d == 0) {
        a.stat[2 * r] = lds.top[h];
        a.stat[2 * r + 1] = l;
      }
    } else {
      const float r = l != l ? l : wk.nt == 0 ? 0.0f : o / l;
      Elem<T>::store(static_cast<T *>(a.o), (static_cast<size_t>(n) * a.Hq + hq + h) * DH + d, r);
    }
  }
}

}  // namespace rglru
