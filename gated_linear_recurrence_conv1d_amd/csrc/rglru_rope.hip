// rglru_rope.hip -- per-head RMS norm of queries and keys with the position rotation in the same
// pass, and its backward (gfx950).
//
// For one head x of dh values (weights w, or none: then n = x) at position t:
//   n_i = x_i r w_i,  r = 1 / sqrt(mean_i x_i^2 + eps),
//   y_i = n_i cos phi_i - n_j sin phi_i,  y_j = n_j cos phi_i + n_i sin phi_i,
//   j = i + rot / 2,  phi_i = t inv_freq_i,  i < rot / 2;  y_i = n_i for i >= rot.
// Backward, with g = (rotation by -phi) dy, xh = x r:
//   dw = sum over rows and heads of g xh,  dx = r (g w - xh mean(g w xh));  dx = g without weights.
//
// phi grows with the position (1e6 turns of the first pair), so the product position * inv_freq
// is formed in fp64 and reduced to a fraction of a turn before it becomes fp32.
//
// Both directions read and write each value once and are bound by memory. A head's values are
// held as chunk pairs: lane c of a head's dh / (2 E) lanes has the 16-byte chunk (E values) of
// pair elements i and the chunk of their partners i + rot / 2, so that the rotation needs no
// exchange, and the norm's sum crosses 4..32 lanes only. A wave works through a run of (row, pass)
// items, a pass being 64 / LPH heads of one row, with the next items' loads in flight (a ring of
// kAhead items: without it a wave waits for memory once per pass, 79 us against 43.5 at B8 T2048 Hq10
// dh256 bf16); a row's angles are formed once for all its passes. Weights and frequencies stay in
// LDS: in registers they would halve the number of waves. There the forward moves its 185 MB at 4.2 TB/s, the
// backward its 277 MB in 53 us, 5.2 TB/s; a plain copy reaches 5.1 TB/s.
#include "rglru_launch.h"
#include "rglru_loads.h"
#include "rglru_mfma.h"

#include <algorithm>

namespace rglru {

namespace {

constexpr double kInvTwoPi = 0.15915494309189533577;

// sin and cos of 2 pi * turns, |turns| <= 1/2. fp32 I/O: the library's sincospi (about an ulp);
// bf16 I/O: the hardware's sine and cosine, whose argument is in turns (error ~1e-6, against the
// output's 2^-9).
template <typename T> __device__ __forceinline__ void sincos_turns(float turns, float &s, float &c) {
  if constexpr (sizeof(T) == 4) {
    sincospif(2.0f * turns, &s, &c);
  } else {
    s = __builtin_amdgcn_sinf(turns);
    c = __builtin_amdgcn_cosf(turns);
  }
}

__device__ __forceinline__ float turns_of(int pos, double freq_turns) {
  const double t = static_cast<double>(pos) * freq_turns;
  return static_cast<float>(t - __builtin_rint(t));
}

// One 16-byte chunk of E values, unpacked to fp32 and back.
template <typename T> struct Chunk;
template <> struct Chunk<bf16_t> {
  static constexpr int E = 8;
  __device__ __forceinline__ static void unpack(u32x4_t v, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16lo(v[i]);
      x[2 * i + 1] = bf16hi(v[i]);
    }
  }
  __device__ __forceinline__ static u32x4_t pack(const float (&x)[E]) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    return v;
  }
};
template <> struct Chunk<float> {
  static constexpr int E = 4;
  __device__ __forceinline__ static void unpack(u32x4_t v, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(v[i]);
  }
  __device__ __forceinline__ static u32x4_t pack(const float (&x)[E]) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(x[i]);
    return v;
  }
};

// Sum over groups of N neighbouring lanes (N a power of two), the result in every lane: within 16
// lanes by data-parallel moves (neighbours, pairs, quads by a half-row mirror, eights by a row
// mirror), beyond by lane exchanges.
template <int CTRL> __device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int N> __device__ __forceinline__ float group_sum(float v) {
  if constexpr (N > 1) v = dpp_add<0xB1>(v);   // quad_perm 1,0,3,2
  if constexpr (N > 2) v = dpp_add<0x4E>(v);   // quad_perm 2,3,0,1
  if constexpr (N > 4) v = dpp_add<0x141>(v);  // row_half_mirror
  if constexpr (N > 8) v = dpp_add<0x140>(v);  // row_mirror
#pragma unroll
  for (int o = 16; o < N; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

constexpr int kRopeWaves = 4;  // waves per workgroup

}  // namespace

// What a lane keeps through all items: its chunk pair's place in a head.
template <typename T, int LPH> struct RopeLane {
  static constexpr int E = Chunk<T>::E;
  static constexpr int HPP = 64 / LPH;  // heads per pass
  static constexpr int DH = 2 * E * LPH;
  int c, hsub, lo, hi;
  bool rotated;
  __device__ __forceinline__ RopeLane(int rot) {
    const int lane = threadIdx.x & 63;
    c = lane % LPH;
    hsub = lane / LPH;
    const int half = rot / 2;
    rotated = c * E < half;
    lo = rotated ? c * E : rot + 2 * (c * E - half);
    hi = rotated ? lo + half : lo + E;
  }
  // sine and cosine of this lane's E angles (0 and 1 where it has none)
  __device__ __forceinline__ void angles(int pos, const double *freq, float (&sn)[E],
                                         float (&cs)[E]) const {
#pragma unroll
    for (int e = 0; e < E; ++e) sincos_turns<T>(turns_of(pos, freq[c * E + e]), sn[e], cs[e]);
  }
};

// Weights (1 without norm) and frequencies in turns (0 beyond rot / 2) to LDS.
template <int DH>
__device__ __forceinline__ void stage_tables(const float *q_w, const float *k_w, const float *inv_freq,
                                             int rot, float (&wl)[2][DH], double (&fl)[DH / 2]) {
  for (int i = threadIdx.x; i < DH; i += 64 * kRopeWaves) {
    wl[0][i] = q_w ? q_w[i] : 1.0f;
    wl[1][i] = q_w ? k_w[i] : 1.0f;
    if (i < DH / 2) fl[i] = i < rot / 2 ? static_cast<double>(inv_freq[i]) * kInvTwoPi : 0.0;
  }
  __syncthreads();
}

constexpr int kAhead = 4;     // items in flight per wave, forward
constexpr int kAheadBwd = 2;  // and backward (twice the loads per item)

// Items (row, pass), pass: heads of q, then of k, then of v on its way to the cache; wave i takes
// items i per .. (i + 1) per - 1.
template <typename T, int LPH>
__global__ __launch_bounds__(64 * kRopeWaves) void qk_rope_fwd(RopeArgs a, int per) {
  typedef RopeLane<T, LPH> L;
  constexpr int E = L::E, HPP = L::HPP, DH = L::DH;
  __shared__ float wl[2][DH];
  __shared__ double fl[DH / 2];
  stage_tables<DH>(a.q_w, a.k_w, a.inv_freq, a.rot, wl, fl);
  const L me(a.rot);
  const bool norm = a.q_w != nullptr;
  const int qp = (a.Hq + HPP - 1) / HPP, kp = (a.Hkv + HPP - 1) / HPP;
  const int passes = qp + kp + (a.slots ? kp : 0);
  const long long items = static_cast<long long>(a.rows) * passes;
  const long long wave = static_cast<long long>(blockIdx.x) * kRopeWaves +
                         __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long f0 = wave * per;
  if (f0 >= items) return;
  const int n = static_cast<int>(min(static_cast<long long>(per), items - f0));
  struct Item {
    u32x4_t lo, hi;
  } ring[kAhead];
  struct At {
    int row, p;
  };
  const int row0 = static_cast<int>(f0 / passes);
  At head = {row0, static_cast<int>(f0 - static_cast<long long>(row0) * passes)}, cur = head;
  auto step = [&](At &at) {
    if (++at.p == passes) {
      at.p = 0;
      ++at.row;
    }
  };
  auto head_of = [&](int p) { return (p < qp ? p : p < qp + kp ? p - qp : p - qp - kp) * HPP + me.hsub; };
  auto load = [&](Item &it) {
    const bool isq = head.p < qp, isv = head.p >= qp + kp;
    const int h = head_of(head.p);
    it.lo = it.hi = u32x4_t{};
    if (h < (isq ? a.Hq : a.Hkv)) {
      const T *src = static_cast<const T *>(isq ? a.q : isv ? a.v : a.k) +
                     static_cast<size_t>(head.row) * (isq ? a.q_stride : isv ? a.v_stride : a.k_stride) +
                     static_cast<size_t>(h) * DH;
      it.lo = *reinterpret_cast<const u32x4_t *>(src + me.lo);
      it.hi = *reinterpret_cast<const u32x4_t *>(src + me.hi);
    }
    step(head);
  };
  int row = -1;
  long long slot = -1;
  float sn[E], cs[E];
  auto process = [&](const Item &it) {
    if (cur.row != row) {
      row = cur.row;
      me.angles(uniform_load(a.positions, row), fl, sn, cs);
      slot = a.slots ? uniform_load(a.slots, row) : -1;
      if (slot >= a.n_slots) slot = -1;
    }
    const bool isq = cur.p < qp, isv = cur.p >= qp + kp;
    const int h = head_of(cur.p);
    const bool on = h < (isq ? a.Hq : a.Hkv);
    step(cur);
    const size_t cache_at =
        (static_cast<size_t>(slot < 0 ? 0 : slot) * a.Hkv + static_cast<size_t>(h)) * DH;
    if (isv) {  // values go to the cache as they are
      if (on && slot >= 0) {
        T *dst = static_cast<T *>(a.v_pages) + cache_at;
        *reinterpret_cast<u32x4_t *>(dst + me.lo) = it.lo;
        *reinterpret_cast<u32x4_t *>(dst + me.hi) = it.hi;
      }
      return;
    }
    float xl[E], xh[E];
    Chunk<T>::unpack(it.lo, xl);
    Chunk<T>::unpack(it.hi, xh);
    if (norm) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) ss = fmaf(xl[e], xl[e], fmaf(xh[e], xh[e], ss));
      ss = group_sum<LPH>(ss);
      const float r = 1.0f / sqrtf(fmaf(ss, 1.0f / DH, a.eps));
      const float *w = wl[isq ? 0 : 1];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xl[e] *= r * w[me.lo + e];
        xh[e] *= r * w[me.hi + e];
      }
    }
    if (me.rotated) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float l = xl[e], g = xh[e];
        xl[e] = l * cs[e] - g * sn[e];
        xh[e] = g * cs[e] + l * sn[e];
      }
    }
    if (!on) return;
    const u32x4_t vl = Chunk<T>::pack(xl), vh = Chunk<T>::pack(xh);
    T *out = static_cast<T *>(isq ? a.q_out : a.k_out);
    if (out) {
      out += static_cast<size_t>(row) * (isq ? a.q_out_stride : a.k_out_stride) +
             static_cast<size_t>(h) * DH;
      *reinterpret_cast<u32x4_t *>(out + me.lo) = vl;
      *reinterpret_cast<u32x4_t *>(out + me.hi) = vh;
    }
    if (!isq && slot >= 0) {
      T *dst = static_cast<T *>(a.k_pages) + cache_at;
      *reinterpret_cast<u32x4_t *>(dst + me.lo) = vl;
      *reinterpret_cast<u32x4_t *>(dst + me.hi) = vh;
    }
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (k < n) load(ring[k]);
  for (int i = 0; i < n; i += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i + k >= n) break;
      const Item it = ring[k];
      if (i + k + kAhead < n) load(ring[k]);
      process(it);
    }
  }
}

// Any even dh <= kRopeMaxDh, any even rot, elements at their natural alignment: one wave per
// (row, head), pair p of the head's dh / 2 in lane p % 64.
constexpr int kRopePairs = kRopeMaxDh / 128;  // pairs per lane
struct PairAt {
  int lo, hi;
};
__device__ __forceinline__ PairAt pair_at(int p, int rot) {
  if (p < rot / 2) return {p, p + rot / 2};
  return {rot + 2 * (p - rot / 2), rot + 2 * (p - rot / 2) + 1};
}

template <typename T>
__global__ __launch_bounds__(64 * kRopeWaves) void qk_rope_fwd_any(RopeArgs a) {
  const int lane = threadIdx.x & 63;
  const int heads = a.Hq + a.Hkv + (a.slots ? a.Hkv : 0);
  const long long tasks = static_cast<long long>(a.rows) * heads;
  const long long nw = static_cast<long long>(gridDim.x) * kRopeWaves;
  const bool norm = a.q_w != nullptr;
  for (long long task = static_cast<long long>(blockIdx.x) * kRopeWaves + (threadIdx.x >> 6);
       task < tasks; task += nw) {
    const int row = static_cast<int>(task / heads);
    const int hh = static_cast<int>(task - static_cast<long long>(row) * heads);
    const bool isq = hh < a.Hq, isv = hh >= a.Hq + a.Hkv;
    const int h = isq ? hh : isv ? hh - a.Hq - a.Hkv : hh - a.Hq;
    const int pos = a.positions[row];
    long long slot = a.slots ? a.slots[row] : -1;
    if (slot >= a.n_slots) slot = -1;
    const size_t cache_at =
        (static_cast<size_t>(slot < 0 ? 0 : slot) * a.Hkv + static_cast<size_t>(h)) * a.dh;
    const T *src = static_cast<const T *>(isq ? a.q : isv ? a.v : a.k) +
                   static_cast<size_t>(row) * (isq ? a.q_stride : isv ? a.v_stride : a.k_stride) +
                   static_cast<size_t>(h) * a.dh;
    float xl[kRopePairs], xh[kRopePairs];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < kRopePairs; ++j) {
      const int p = lane + 64 * j;
      xl[j] = xh[j] = 0.0f;
      if (2 * p < a.dh) {
        const PairAt at = pair_at(p, a.rot);
        xl[j] = Elem<T>::load(src, at.lo);
        xh[j] = Elem<T>::load(src, at.hi);
      }
      ss = fmaf(xl[j], xl[j], fmaf(xh[j], xh[j], ss));
    }
    if (isv) {
      if (slot >= 0) {
        T *dst = static_cast<T *>(a.v_pages) + cache_at;
#pragma unroll
        for (int j = 0; j < kRopePairs; ++j) {
          const int p = lane + 64 * j;
          if (2 * p < a.dh) {
            const PairAt at = pair_at(p, a.rot);
            Elem<T>::store(dst, at.lo, xl[j]);
            Elem<T>::store(dst, at.hi, xh[j]);
          }
        }
      }
      continue;
    }
    const float *w = isq ? a.q_w : a.k_w;
    float r = 1.0f;
    if (norm) r = 1.0f / sqrtf(fmaf(group_sum<64>(ss), 1.0f / static_cast<float>(a.dh), a.eps));
    T *out = static_cast<T *>(isq ? a.q_out : a.k_out);
    if (out)
      out += static_cast<size_t>(row) * (isq ? a.q_out_stride : a.k_out_stride) +
             static_cast<size_t>(h) * a.dh;
    T *dst = !isq && slot >= 0 ? static_cast<T *>(a.k_pages) + cache_at : nullptr;
#pragma unroll
    for (int j = 0; j < kRopePairs; ++j) {
      const int p = lane + 64 * j;
      if (2 * p >= a.dh) continue;
      const PairAt at = pair_at(p, a.rot);
      float l = xl[j], g = xh[j];
      if (norm) {
        l *= r * w[at.lo];
        g *= r * w[at.hi];
      }
      if (p < a.rot / 2) {
        float s, c;
        sincos_turns<float>(turns_of(pos, static_cast<double>(a.inv_freq[p]) * kInvTwoPi), s, c);
        const float l0 = l;
        l = l0 * c - g * s;
        g = g * c + l0 * s;
      }
      if (out) {
        Elem<T>::store(out, at.lo, l);
        Elem<T>::store(out, at.hi, g);
      }
      if (dst) {
        Elem<T>::store(dst, at.lo, l);
        Elem<T>::store(dst, at.hi, g);
      }
    }
  }
}

// Backward. Items and waves as in the forward (no cache passes), but a pass may hold heads of q and of k: kept
// apart, a single key head fills a quarter of its pass at dh 256 (71 us against 60 at B8 T2048 Hq10 bf16; in the
// forward, whose lanes then choose between three sources and outputs, 43.4 against 44.2). A wave keeps the weights' gradients
// of its chunk columns in registers; a workgroup writes one partial row, part[blockIdx.x][2][dh] (q,
// k), and rope_dw_sum adds the rows in order. The grid depends on the sizes alone, so the sums are
// bitwise reproducible.
template <typename T, int LPH>
__global__ __launch_bounds__(64 * kRopeWaves, 3) void qk_rope_bwd(RopeBwdArgs a, int per) {
  typedef RopeLane<T, LPH> L;
  constexpr int E = L::E, HPP = L::HPP, DH = L::DH;
  __shared__ float wl[2][DH];
  __shared__ double fl[DH / 2];
  __shared__ float red[kRopeWaves][2][DH];
  stage_tables<DH>(a.q_w, a.k_w, a.inv_freq, a.rot, wl, fl);
  const L me(a.rot);
  const bool norm = a.q_w != nullptr;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int heads = a.Hq + a.Hkv, passes = (heads + HPP - 1) / HPP;
  const long long items = static_cast<long long>(a.rows) * passes;
  const long long f0 = min(items, (static_cast<long long>(blockIdx.x) * kRopeWaves + w) * per);
  const int n = static_cast<int>(min(static_cast<long long>(per), items - f0));
  struct Item {
    u32x4_t gl, gh, xl, xh;
  } ring[kAheadBwd];
  struct At {
    int row, p;
  };
  const int row0 = static_cast<int>(f0 / passes);
  At head = {row0, static_cast<int>(f0 - static_cast<long long>(row0) * passes)}, cur = head;
  auto step = [&](At &at) {
    if (++at.p == passes) {
      at.p = 0;
      ++at.row;
    }
  };
  auto load = [&](Item &it) {
    const int hh = head.p * HPP + me.hsub;
    it.gl = it.gh = it.xl = it.xh = u32x4_t{};
    if (hh < heads) {
      const bool isq = hh < a.Hq;
      const size_t hoff = static_cast<size_t>(isq ? hh : hh - a.Hq) * DH;
      const T *g = static_cast<const T *>(isq ? a.dq_out : a.dk_out) +
                   static_cast<size_t>(head.row) * (isq ? a.dq_out_stride : a.dk_out_stride) + hoff;
      it.gl = *reinterpret_cast<const u32x4_t *>(g + me.lo);
      it.gh = *reinterpret_cast<const u32x4_t *>(g + me.hi);
      if (norm) {
        const T *x = static_cast<const T *>(isq ? a.q : a.k) +
                     static_cast<size_t>(head.row) * (isq ? a.q_stride : a.k_stride) + hoff;
        it.xl = *reinterpret_cast<const u32x4_t *>(x + me.lo);
        it.xh = *reinterpret_cast<const u32x4_t *>(x + me.hi);
      }
    }
    step(head);
  };
  float aq[2 * E] = {}, ak[2 * E] = {};
  int row = -1;
  float sn[E], cs[E];
  auto grad = [&](const Item &it, bool isq, float (&dl)[E], float (&dh)[E]) {
    Chunk<T>::unpack(it.gl, dl);
    Chunk<T>::unpack(it.gh, dh);
    if (me.rotated) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float l = dl[e], q = dh[e];
        dl[e] = l * cs[e] + q * sn[e];
        dh[e] = q * cs[e] - l * sn[e];
      }
    }
    if (!norm) return;
    const float *wt = wl[isq ? 0 : 1];
    float xl[E], xh[E];
    Chunk<T>::unpack(it.xl, xl);
    Chunk<T>::unpack(it.xh, xh);
    float ss = 0.0f, st = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      ss = fmaf(xl[e], xl[e], fmaf(xh[e], xh[e], ss));
      st = fmaf(dl[e] * wt[me.lo + e], xl[e], fmaf(dh[e] * wt[me.hi + e], xh[e], st));
    }
    ss = group_sum<LPH>(ss);
    st = group_sum<LPH>(st);
    const float r = 1.0f / sqrtf(fmaf(ss, 1.0f / DH, a.eps));
    const float m = st * r * (1.0f / DH);  // mean(g w xh)
    // (by branch, not by a zero factor: what is not finite in a head of k stays out of q's sums)
    if (isq) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        aq[e] = fmaf(dl[e], xl[e] * r, aq[e]);
        aq[E + e] = fmaf(dh[e], xh[e] * r, aq[E + e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        ak[e] = fmaf(dl[e], xl[e] * r, ak[e]);
        ak[E + e] = fmaf(dh[e], xh[e] * r, ak[E + e]);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float nl = xl[e] * r, nh = xh[e] * r;
      dl[e] = r * fmaf(-nl, m, dl[e] * wt[me.lo + e]);
      dh[e] = r * fmaf(-nh, m, dh[e] * wt[me.hi + e]);
    }
  };
  auto process = [&](const Item &it) {
    if (cur.row != row) {
      row = cur.row;
      me.angles(uniform_load(a.positions, row), fl, sn, cs);
    }
    const int hh = cur.p * HPP + me.hsub;
    const bool isq = hh < a.Hq;
    step(cur);
    float dl[E], dh[E];
    grad(it, isq, dl, dh);
    if (hh < heads) {
      T *d = static_cast<T *>(isq ? a.dq : a.dk) + static_cast<size_t>(row) * (isq ? a.dq_stride : a.dk_stride) +
             static_cast<size_t>(isq ? hh : hh - a.Hq) * DH;
      *reinterpret_cast<u32x4_t *>(d + me.lo) = Chunk<T>::pack(dl);
      *reinterpret_cast<u32x4_t *>(d + me.hi) = Chunk<T>::pack(dh);
    }
  };
#pragma unroll
  for (int k = 0; k < kAheadBwd; ++k)
    if (k < n) load(ring[k]);
  for (int i = 0; i < n; i += kAheadBwd) {
#pragma unroll
    for (int k = 0; k < kAheadBwd; ++k) {
      if (i + k >= n) break;
      const Item it = ring[k];
      if (i + k + kAheadBwd < n) load(ring[k]);
      process(it);
    }
  }
  if (!norm) return;
  // the wave's head groups (lanes c, c + LPH, ..), then the workgroup's waves
#pragma unroll
  for (int e = 0; e < 2 * E; ++e) {
#pragma unroll
    for (int o = LPH; o < 64; o <<= 1) {
      aq[e] += __shfl_xor(aq[e], o, 64);
      ak[e] += __shfl_xor(ak[e], o, 64);
    }
  }
  if (me.hsub == 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      red[w][0][me.lo + e] = aq[e];
      red[w][0][me.hi + e] = aq[E + e];
      red[w][1][me.lo + e] = ak[e];
      red[w][1][me.hi + e] = ak[E + e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * DH; i += 64 * kRopeWaves) {
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kRopeWaves; ++v) s += (&red[v][0][0])[i];
    a.part[static_cast<size_t>(blockIdx.x) * 2 * DH + i] = s;
  }
}

template <typename T>
__global__ __launch_bounds__(64 * kRopeWaves) void qk_rope_bwd_any(RopeBwdArgs a) {
  __shared__ float red[kRopeWaves][2][kRopeMaxDh];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const bool norm = a.q_w != nullptr;
  float acc[2][kRopePairs][2] = {};
  const long long nw = static_cast<long long>(gridDim.x) * kRopeWaves;
  for (long long row = static_cast<long long>(blockIdx.x) * kRopeWaves + w; row < a.rows; row += nw) {
    const int pos = a.positions[row];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const bool isq = kind == 0;
      const float *wt = isq ? a.q_w : a.k_w;
      for (int h = 0; h < (isq ? a.Hq : a.Hkv); ++h) {
        const size_t hoff = static_cast<size_t>(h) * a.dh;
        const T *g = static_cast<const T *>(isq ? a.dq_out : a.dk_out) +
                     static_cast<size_t>(row) * (isq ? a.dq_out_stride : a.dk_out_stride) + hoff;
        const T *x = static_cast<const T *>(isq ? a.q : a.k) +
                     static_cast<size_t>(row) * (isq ? a.q_stride : a.k_stride) + hoff;
        T *d = static_cast<T *>(isq ? a.dq : a.dk) +
               static_cast<size_t>(row) * (isq ? a.dq_stride : a.dk_stride) + hoff;
        float gl[kRopePairs], gh[kRopePairs], xl[kRopePairs], xh[kRopePairs];
        float ss = 0.0f, st = 0.0f;
#pragma unroll
        for (int j = 0; j < kRopePairs; ++j) {
          const int p = lane + 64 * j;
          gl[j] = gh[j] = xl[j] = xh[j] = 0.0f;
          if (2 * p >= a.dh) continue;
          const PairAt at = pair_at(p, a.rot);
          gl[j] = Elem<T>::load(g, at.lo);
          gh[j] = Elem<T>::load(g, at.hi);
          if (p < a.rot / 2) {
            float s, c;
            sincos_turns<float>(turns_of(pos, static_cast<double>(a.inv_freq[p]) * kInvTwoPi), s, c);
            const float l0 = gl[j];
            gl[j] = l0 * c + gh[j] * s;
            gh[j] = gh[j] * c - l0 * s;
          }
          if (norm) {
            xl[j] = Elem<T>::load(x, at.lo);
            xh[j] = Elem<T>::load(x, at.hi);
            ss = fmaf(xl[j], xl[j], fmaf(xh[j], xh[j], ss));
            st = fmaf(gl[j] * wt[at.lo], xl[j], fmaf(gh[j] * wt[at.hi], xh[j], st));
          }
        }
        float r = 1.0f, m = 0.0f;
        if (norm) {
          const float inv = 1.0f / static_cast<float>(a.dh);
          r = 1.0f / sqrtf(fmaf(group_sum<64>(ss), inv, a.eps));
          m = group_sum<64>(st) * r * inv;
        }
#pragma unroll
        for (int j = 0; j < kRopePairs; ++j) {
          const int p = lane + 64 * j;
          if (2 * p >= a.dh) continue;
          const PairAt at = pair_at(p, a.rot);
          float dl = gl[j], dh = gh[j];
          if (norm) {
            const float nl = xl[j] * r, nh = xh[j] * r;
            acc[kind][j][0] = fmaf(gl[j], nl, acc[kind][j][0]);
            acc[kind][j][1] = fmaf(gh[j], nh, acc[kind][j][1]);
            dl = r * fmaf(-nl, m, gl[j] * wt[at.lo]);
            dh = r * fmaf(-nh, m, gh[j] * wt[at.hi]);
          }
          Elem<T>::store(d, at.lo, dl);
          Elem<T>::store(d, at.hi, dh);
        }
      }
    }
  }
  if (!norm) return;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int j = 0; j < kRopePairs; ++j) {
      const int p = lane + 64 * j;
      if (2 * p >= a.dh) continue;
      const PairAt at = pair_at(p, a.rot);
      red[w][kind][at.lo] = acc[kind][j][0];
      red[w][kind][at.hi] = acc[kind][j][1];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.dh; i += 64 * kRopeWaves) {
    const int kind = i / a.dh, d = i - kind * a.dh;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kRopeWaves; ++v) s += red[v][kind][d];
    a.part[static_cast<size_t>(blockIdx.x) * 2 * a.dh + i] = s;
  }
}

// dq_w, dk_w = the sums of part's rows: one workgroup per 32 columns, 32 row groups of 32 lanes,
// each group its rows in order, then the groups in order.
__global__ __launch_bounds__(1024) void rope_dw_sum(const float *part, int rows, int dh,
                                                    float *dq_w, float *dk_w) {
  __shared__ float red[32][33];
  const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + col;
  float s = 0.0f;
  if (i < 2 * dh) {
#pragma unroll 8
    for (int r = grp; r < rows; r += 32) s += part[static_cast<size_t>(r) * 2 * dh + i];
  }
  red[grp][col] = s;
  __syncthreads();
  if (grp == 0 && i < 2 * dh) {
    float t = 0.0f;
#pragma unroll
    for (int g = 0; g < 32; ++g) t += red[g][col];
    if (i < dh)
      dq_w[i] = t;
    else
      dk_w[i - dh] = t;
  }
}

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The chunk-pair kernels: dh in {64, 128, 256}, rot in whole chunk pairs, every address a
// multiple of 16 bytes.
bool chunked(int dh, int rot, int io, const void *const *ptrs, int np, const long long *strides,
             int ns) {
  const int e = io == kBF16 ? 8 : 4;
  if ((dh != 64 && dh != 128 && dh != 256) || rot % (2 * e)) return false;
  for (int i = 0; i < np; ++i)
    if (!aligned16(ptrs[i])) return false;
  for (int i = 0; i < ns; ++i)
    if (strides[i] % e) return false;
  return true;
}

}  // namespace

namespace {

// Items of one wave: enough waves for the chip, whole rows once a wave has more than one (a row's
// angles are then formed once).
constexpr long long kFwdWaves = 8192;
int items_per_wave(int rows, int passes, long long waves) {
  const long long items = static_cast<long long>(rows) * passes;
  const long long per = (items + waves - 1) / waves;
  return static_cast<int>(per <= 1 ? 1 : (per + passes - 1) / passes * passes);
}

}  // namespace

hipError_t launch_qk_rope(const RopeArgs &a, int io, hipStream_t s) {
  const void *ptrs[] = {a.q, a.k, a.v, a.q_out, a.k_out, a.k_pages, a.v_pages};
  const long long st[] = {a.q_stride, a.k_stride, a.v ? a.v_stride : 0, a.q_out_stride,
                          a.k_out ? a.k_out_stride : 0};
  const int kThr = 64 * kRopeWaves;
  if (!chunked(a.dh, a.rot, io, ptrs, 7, st, 5)) {
    const long long tasks = static_cast<long long>(a.rows) * (a.Hq + a.Hkv * (a.slots ? 2 : 1));
    const unsigned grid = static_cast<unsigned>(
        std::min<long long>((tasks + kRopeWaves - 1) / kRopeWaves, 1 << 14));
    if (io == kBF16)
      qk_rope_fwd_any<bf16_t><<<grid, kThr, 0, s>>>(a);
    else
      qk_rope_fwd_any<float><<<grid, kThr, 0, s>>>(a);
    return hipGetLastError();
  }
  const int lph = a.dh / (io == kBF16 ? 16 : 8), hpp = 64 / lph;
  const int kp = (a.Hkv + hpp - 1) / hpp;
  const int passes = (a.Hq + hpp - 1) / hpp + kp + (a.slots ? kp : 0);
  const int per = items_per_wave(a.rows, passes, kFwdWaves);
  const long long waves = (static_cast<long long>(a.rows) * passes + per - 1) / per;
  const unsigned grid = static_cast<unsigned>((waves + kRopeWaves - 1) / kRopeWaves);
  if (io == kBF16) {
    switch (a.dh) {
      case 64: qk_rope_fwd<bf16_t, 4><<<grid, kThr, 0, s>>>(a, per); break;
      case 128: qk_rope_fwd<bf16_t, 8><<<grid, kThr, 0, s>>>(a, per); break;
      default: qk_rope_fwd<bf16_t, 16><<<grid, kThr, 0, s>>>(a, per); break;
    }
  } else {
    switch (a.dh) {
      case 64: qk_rope_fwd<float, 8><<<grid, kThr, 0, s>>>(a, per); break;
      case 128: qk_rope_fwd<float, 16><<<grid, kThr, 0, s>>>(a, per); break;
      default: qk_rope_fwd<float, 32><<<grid, kThr, 0, s>>>(a, per); break;
    }
  }
  return hipGetLastError();
}

int rope_bwd_groups(int rows) {
  return std::min((rows + kRopeWaves - 1) / kRopeWaves, 768);  // three a CU, all there at once (1024: 60 us for 53)
}

hipError_t launch_qk_rope_backward(const RopeBwdArgs &a, float *dq_w, float *dk_w, int io,
                                   hipStream_t s) {
  const void *ptrs[] = {a.q, a.k, a.dq_out, a.dk_out, a.dq, a.dk};
  const long long st[] = {a.q_stride,      a.k_stride,  a.dq_out_stride,
                          a.dk_out_stride, a.dq_stride, a.dk_stride};
  const int kThr = 64 * kRopeWaves;
  const unsigned grid = static_cast<unsigned>(rope_bwd_groups(a.rows));
  const int hpp = 64 / std::max(1, a.dh / (io == kBF16 ? 16 : 8));
  const int passes = hpp < 1 ? 1 : (a.Hq + a.Hkv + hpp - 1) / hpp;
  const long long items = static_cast<long long>(a.rows) * passes, waves = static_cast<long long>(grid) * kRopeWaves;
  const int per = static_cast<int>((items + waves - 1) / waves);
  if (!chunked(a.dh, a.rot, io, ptrs, 6, st, 6)) {
    if (io == kBF16)
      qk_rope_bwd_any<bf16_t><<<grid, kThr, 0, s>>>(a);
    else
      qk_rope_bwd_any<float><<<grid, kThr, 0, s>>>(a);
  } else if (io == kBF16) {
    switch (a.dh) {
      case 64: qk_rope_bwd<bf16_t, 4><<<grid, kThr, 0, s>>>(a, per); break;
      case 128: qk_rope_bwd<bf16_t, 8><<<grid, kThr, 0, s>>>(a, per); break;
      default: qk_rope_bwd<bf16_t, 16><<<grid, kThr, 0, s>>>(a, per); break;
    }
  } else {
    switch (a.dh) {
      case 64: qk_rope_bwd<float, 8><<<grid, kThr, 0, s>>>(a, per); break;
      case 128: qk_rope_bwd<float, 16><<<grid, kThr, 0, s>>>(a, per); break;
      default: qk_rope_bwd<float, 32><<<grid, kThr, 0, s>>>(a, per); break;
    }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.q_w) return e;
  rope_dw_sum<<<(2 * a.dh + 31) / 32, 1024, 0, s>>>(a.part, static_cast<int>(grid), a.dh, dq_w, dk_w);
  return hipGetLastError();
}

}  // namespace rglru
