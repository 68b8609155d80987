// rglru_attn.hip -- local attention with grouped heads, sinks, a length per sequence and strided tokens,
// forward, bf16 on gfx950 (rglru_local_attention).
//
//   o[t] = sum_u p_u v_u,  p_u = exp(scale s_u - lse),  s_u = <q_t, k_u>,
//   u <= t and (u > t - W or u < sinks), t and u below the sequence's length.
//
// One pass over the visible keys with a running maximum m and sum l per row. Both contractions put a
// query row in each lane: S^T = K Q^T (A = K rows from LDS, B = q in registers for the kernel's life) and
// O^T += V^T P^T (A = V^T from LDS by transposing reads, B = P). The accumulator layout of S^T is already the
// B operand's of the second, so P never leaves its lane. A wave owns 32 rows and all of dh (64 registers of q
// and 128 of O at dh 256: two waves per SIMD); four waves are a workgroup, two or three workgroups share a
// CU, and each wave works alone between the barriers (one per 32-key block), so that one wave's matrix
// work runs beside another's exponentials.
//
// Bound at dh 128 by the matrix and vector units in turn, which overlap only across the two or three waves of a SIMD
// (busy 37% and 39% of the cycles, CUs 75%); at dh 256 by the waits between a wave's steps beside them (31% and 27%
// of 75%). LDS is busy 17-19%. 96 us at B8 T2048 (ragged) Hq10 dh256 W1024 (670 TFLOP/s), 310 us at T16384 Hq8 Hkv2
// dh128 W4096 (780 TFLOP/s).
#include "rglru_attn.h"
#include "rglru_grid.h"
#include "rglru_launch.h"

#include <algorithm>
#include <type_traits>

namespace rglru {

using namespace attn;

namespace {

// P enters P V as bf16 hi + lo in workgroups where some row sees fewer keys: there the rounding of P to
// bf16 does not average out (a row's worst element then stays near 4e-3 of the output's rms instead of
// up to 4e-2; with 256 keys or more bf16 alone is below 9e-3)
constexpr int kSplitKeys = 256;
// s c - m c in one FMA is off by the rounding of m c, 2^-24 of it: for scores beyond this (in exp2
// units) the difference s - m is formed first
constexpr float kBigScore = 16384.0f;
constexpr int kAhead = 3;  // MFMA steps that LDS operands are read ahead

}  // namespace

// o of one row from the definition alone, one key at a time (DH / 64 values of every row per lane).
// Only for rows whose o came out non-finite although their scores are finite: the tile's P V adds
// 0 * v for the keys that a row does not see, which is not 0 where v is infinite or NaN.
template <int DH>
__device__ __forceinline__ void exact_row(const bf16_t *q, const bf16_t *k, const bf16_t *v, bf16_t *o,
                                          const AttnArgs &x, float c, int t, int lane) {
  constexpr int kPer = DH / 64;
  float qv[kPer], a[kPer] = {};
#pragma unroll
  for (int i = 0; i < kPer; ++i) qv[i] = bf16_to_f32(q[lane * kPer + i]);
  float m = x.floor, l = 0.0f;
  const int lo = max(0, t - x.window + 1);
  for (int u = x.sinks > 0 ? 0 : lo; u <= t;) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      s = fmaf(qv[i], bf16_to_f32(k[static_cast<size_t>(u) * x.k_stride + lane * kPer + i]), s);
#pragma unroll
    for (int e = 1; e < 64; e <<= 1) s += __shfl_xor(s, e, 64);
    const float mn = fmaxf(m, s);
    const float corr = __builtin_amdgcn_exp2f((m - mn) * c);
    const float p = __builtin_amdgcn_exp2f((s - mn) * c);
    m = mn;
    l = l * corr + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      a[i] = a[i] * corr + p * bf16_to_f32(v[static_cast<size_t>(u) * x.v_stride + lane * kPer + i]);
    bool done = true;  // all of o is NaN already
#pragma unroll
    for (int i = 0; i < kPer; ++i) done = done && a[i] != a[i];
    if (__all(done)) break;
    ++u;
    if (u == x.sinks && u < lo) u = lo;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[lane * kPer + i] = f32_to_bf16(a[i] / l);
}

// KS: groups of four waves that share the rows, each with every KS-th key block, joined at the end.
template <int DH, int KS>
__global__ __launch_bounds__(64 * kWg * KS, 2) void attn_fwd(AttnArgs x) {
  typedef Blk<DH> K;
  constexpr int kRows = kOwn;  // per workgroup
  __shared__ __attribute__((aligned(1024))) unsigned char smem[KS * 2 * K::kSlot];  // two slots of K, V a group
  __shared__ float joined[KS > 1 ? 2 : 1][KS > 1 ? 64 * kWg : 1];                   // group 1's m and l
  static_assert(KS <= 2 && (KS == 1 || sizeof(smem) >= kRows * DH * sizeof(float)), "room for group 1's O");
  const int tid = threadIdx.x, lane = tid & 63;
  const int grp = KS > 1 ? uni(tid >> 6) / kWg : 0, w = uni(tid >> 6) - grp * kWg;
  const unsigned lds = lds_addr(smem) + grp * 2 * K::kSlot;
  const int lrow = lane & 31, half = lane >> 5;
  const int T = x.T, Hq = x.Hq, W = x.window, sinks = x.sinks;
  const float c = x.scale * kLn2Inv;
  // heavy first: query blocks from the last one down, all (sequence, head) pairs of one together
  const int nbh = x.B * Hq, nqb = (T + kRows - 1) / kRows;
  const int id = block_of(blockIdx.y);
  const int qi = uni(id / nbh), bh = id - qi * nbh;
  if (qi >= nqb) return;
  const int q0 = (nqb - 1 - qi) * kRows;
  const int b = uni(bh / Hq), h = bh - b * Hq;
  const int kvh = uni(h / (Hq / x.Hkv));
  const int len = clamp_len(x.lens, b, T);
  const size_t tok = static_cast<size_t>(b) * T;
  const size_t ostride = static_cast<size_t>(Hq) * DH;
  bf16_t *const o_ = static_cast<bf16_t *>(x.o) + tok * ostride + static_cast<size_t>(h) * DH;
  float *const lse_ = x.lse ? x.lse + (static_cast<size_t>(b) * Hq + h) * T : nullptr;
  if (q0 >= len) {  // no row of the block belongs to the sequence
    for (int i = tid; i < kRows * (DH / 8); i += 64 * kWg * KS) {
      const int t = q0 + i / (DH / 8);
      if (t < T) *reinterpret_cast<u32x4_t *>(o_ + static_cast<size_t>(t) * ostride + (i % (DH / 8)) * 8) = u32x4_t{};
    }
    for (int i = tid; lse_ && i < kRows; i += 64 * kWg * KS)
      if (q0 + i < T) lse_[q0 + i] = -__builtin_inff();
    return;
  }
  const int qw = q0 + 32 * w, qr = qw + lrow;  // this wave's first row, this lane's row
  const bf16_t *const q_ = static_cast<const bf16_t *>(x.q) + tok * x.q_stride + static_cast<size_t>(h) * DH;
  const bf16_t *const k_ = static_cast<const bf16_t *>(x.k) + tok * x.k_stride + static_cast<size_t>(kvh) * DH;
  const bf16_t *const v_ = static_cast<const bf16_t *>(x.v) + tok * x.v_stride + static_cast<size_t>(kvh) * DH;
  bf16x8_t qf[K::kKS];
  const unsigned tile = lds + w * K::kBytes;  // this wave's, before and after the walk
  Tile<DH>::start(q_ + static_cast<size_t>(qw) * x.q_stride, static_cast<unsigned>(x.q_stride) * 2, len - qw, lane,
                  tile);
  Tile<DH>::landed();
#pragma unroll
  for (int s = 0; s < K::kKS; ++s) qf[s] = Tile<DH>::operand(tile, lane, s);
  lds_barrier();  // everyone has its rows: the slots may be filled
  const BlockWalk walk(q0, kRows, len, W, sinks);
  const unsigned krb = static_cast<unsigned>(x.k_stride) * 2, vrb = static_cast<unsigned>(x.v_stride) * 2;
  const typename K::Lane kl = K::load_lane(w, lane, krb), vl = K::load_lane(w, lane, vrb);
  // the rows of the group's i-th block (past the last one: none, which reads zeros without touching memory)
  struct Src {
    __amdgpu_buffer_rsrc_t k, v;
    unsigned dst;
  };
  auto src_of = [&](int i) {
    const int n = KS * i + grp, u0 = walk.first_row(min(n, walk.n - 1)), rows = n < walk.n ? len - u0 : 0;
    return Src{K::rsrc(k_ + static_cast<size_t>(u0) * x.k_stride, krb, rows),
               K::rsrc(v_ + static_cast<size_t>(u0) * x.v_stride, vrb, rows), lds + (i & 1) * K::kSlot};
  };
  // the n-th of this wave's 2 kLPW loads of a block, of K and V in turn
  auto load_part = [&](const Src &src, int n) {
    if (n % 2 == 0)
      K::load(src.k, krb, n / 2, w, kl, src.dst);
    else
      K::load(src.v, vrb, n / 2, w, vl, src.dst + K::kBytes);
  };
  auto load_block = [&](const Src &src) {
#pragma unroll
    for (int n = 0; n < 2 * K::kLPW; ++n) load_part(src, n);
  };
  const unsigned row_lane = K::row_lane(lane), col_lane = K::col_lane(lane);

  unsigned odd = 0;  // rows to do again
  // the whole walk and the stores, P as bf16 (kSplit: as bf16 hi + lo)
  auto run = [&](auto split_c) {
    constexpr bool kSplit = decltype(split_c)::value;
    f32x16_t acc[K::kDT];  // O^T
#pragma unroll
    for (int j = 0; j < K::kDT; ++j) acc[j] = f32x16_t{};
    float m = x.floor, l = 0.0f;  // running maximum (of raw scores), and this half's sum
    load_block(src_of(0));
    for (int i = 0; i < (walk.n + KS - 1) / KS; ++i) {
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's rows of block i landed
      lds_barrier();                        // everyone's landed; everyone is done with block i - 1
      const int U = walk.first_row(KS * i + grp);
      const bool vis = (KS == 1 || KS * i + grp < walk.n) && U <= qw + 31 && (U + 31 > qw - W || U < sinks) && qw < len;
      // the next block's loads: between the MFMAs, or at once in a wave that sees nothing of this block
      // (that branch kept apart from the next one: as its else, it costs registers)
      int burst = vis ? 0 : 1;
      asm volatile("" : "+v"(burst));
      const Src src = src_of(i + 1);
      if (uni(burst)) load_block(src);
      if (!vis) continue;
      const unsigned slot = lds + (i & 1) * K::kSlot;
      // S^T: K rows read kAhead steps ahead, pinned by the scheduling barriers (the compiler else reads each
      // right before its use)
      // the matrix work goes first: where a wave's turn comes between another's exponentials, both run (98 us
      // with this, 106 without, at B8 T2048 Hq10 dh256 W1024)
      __builtin_amdgcn_s_setprio(1);
      f32x16_t s = f32x16_t{};
      {
        unsigned ks = slot + row_lane;
        asm volatile("" : "+v"(ks));
        bf16x8_t kr[kAhead + 1];
#pragma unroll
        for (int d = 0; d < kAhead; ++d) kr[d] = K::rows(ks, d);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < K::kKS; ++d) {
          if (d + kAhead < K::kKS) kr[(d + kAhead) % (kAhead + 1)] = K::rows(ks, d + kAhead);
          if (d % 2 == 0) load_part(src, d / 2);
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kr[d % (kAhead + 1)], qf[d], s, 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_s_setprio(0);
      const bool full = U + 31 <= qw && (U > qw + 31 - W || U + 31 < sinks) && U + 31 < len;
      if (!full) {
        // (lane terms from the thread index here: kept, they would take registers from the whole walk)
        const int tx = static_cast<int>(__builtin_amdgcn_workitem_id_x());
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int u = U + 8 * (e >> 2) + 4 * ((tx >> 5) & 1) + (e & 3);
          s[e] = sees(qw + (tx & 31), u, W, sinks) && u < len ? s[e] : -__builtin_inff();
        }
      }
      float mx = fmaxf(s[0], s[1]), my = fmaxf(s[2], s[3]);
#pragma unroll
      for (int e = 4; e < 16; e += 2) {
        mx = fmaxf(mx, s[e]);
        my = fmaxf(my, s[e + 1]);
      }
      float lo, hi;
      halves(fmaxf(mx, my), lo, hi);
      mx = fmaxf(fmaxf(lo, hi), x.floor);
      // O and l are kept relative to a maximum that is raised only when a row's grows by more than 2^8:
      // they share it, so the result does not change, and the rescale is rare
      const bool raise = (mx - m) * c > 8.0f;
      if (__any(raise)) {
        const float mn = raise ? mx : m;
        const float corr = __builtin_amdgcn_exp2f((m - mn) * c);
        l *= corr;
        m = mn;
#pragma unroll
        for (int j = 0; j < K::kDT; ++j) acc[j] *= corr;
      }
      const float mc = m * c;
      if (__any(fabsf(mc) > kBigScore)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = (s[e] - m) * c;
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = fmaf(s[e], c, -mc);
      }
      u32x4_t p[2], pl[2];  // P of two 16-key steps, hi (and lo)
      float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float a = __builtin_amdgcn_exp2f(s[e]), bb = __builtin_amdgcn_exp2f(s[e + 1]);
        l0 += a;
        l1 += bb;
        const uint32_t hw = pack_bf16x2(a, bb);
        p[e >> 3][(e >> 1) & 3] = hw;
        if constexpr (kSplit) pl[e >> 3][(e >> 1) & 3] = pack_bf16x2(a - bf16lo(hw), bb - bf16hi(hw));
      }
      l += l0 + l1;
      __builtin_amdgcn_s_setprio(1);
      // O^T += V^T P^T: step n is key step n / kDT, d tile n % kDT
      {
        unsigned vs = slot + K::kBytes + col_lane;
        asm volatile("" : "+v"(vs));  // one register; the steps' XORs are then with literals
        auto v_of = [&](int n) { return K::cols(vs, n & 1, n >> 1); };
        bf16x8_t vt[kAhead + 1];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) vt[n] = v_of(n);
#pragma unroll
        for (int n = 0; n < 2 * K::kDT; ++n) {
          if (n + kAhead < 2 * K::kDT) vt[(n + kAhead) % (kAhead + 1)] = v_of(n + kAhead);
          f32x16_t &o = acc[n >> 1];
          o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              vt[n % (kAhead + 1)], __builtin_bit_cast(bf16x8_t, p[n & 1]), o, 0, 0, 0);
          if constexpr (kSplit)
            o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                vt[n % (kAhead + 1)], __builtin_bit_cast(bf16x8_t, pl[n & 1]), o, 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_s_setprio(0);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // the zeros past the last block have landed too
    lds_barrier();                        // everyone is done with the slots
    if constexpr (KS > 1) {
      f32x4_t *const o1 = reinterpret_cast<f32x4_t *>(smem) + w * 64 + lane;  // in the accumulators' order
      if (grp == 1) {
#pragma unroll
        for (int j = 0; j < K::kDT; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            o1[(4 * j + g) * 64 * kWg] = f32x4_t{acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
        joined[0][w * 64 + lane] = m;
        joined[1][w * 64 + lane] = l;
      }
      lds_barrier();
      if (grp == 0) {
        const float m1 = joined[0][w * 64 + lane], mn = fmaxf(m, m1);
        const float f0 = __builtin_amdgcn_exp2f((m - mn) * c), f1 = __builtin_amdgcn_exp2f((m1 - mn) * c);
        l = l * f0 + joined[1][w * 64 + lane] * f1;
        m = mn;
#pragma unroll
        for (int j = 0; j < K::kDT; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4_t y = o1[(4 * j + g) * 64 * kWg];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][4 * g + e] = acc[j][4 * g + e] * f0 + y[e] * f1;
          }
      }
      lds_barrier();
      if (grp != 0) return;
    }
    // normalise and store; lane = row, accumulator e of tile j is d = 32 j + 8 (e / 4) + 4 half + e % 4
    float lo, hi;
    halves(l, lo, hi);
    const float lt = lo + hi;
    const bool in = qr < len;
    const float inv = 1.0f / lt;
    float worst = 0.0f;
#pragma unroll
    for (int j = 0; j < K::kDT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        acc[j][e] = in ? acc[j][e] * inv : 0.0f;
        worst = fmaf(0.0f, acc[j][e], worst);  // NaN if any is not finite
      }
    Tile<DH>::store(
        tile, lane,
        [&](int j, int g) {
          return u32x2_t{pack_bf16x2(acc[j][4 * g], acc[j][4 * g + 1]),
                         pack_bf16x2(acc[j][4 * g + 2], acc[j][4 * g + 3])};
        },
        o_ + static_cast<size_t>(qw) * ostride, ostride, T - qw);
    // ln of the denominator sum_u exp(scale s_u) = scale m + ln l
    if (lse_ && half == 0 && qr < T)
      lse_[qr] = in ? (m * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f : -__builtin_inff();
    const unsigned long long rows = __ballot(in && !(worst == 0.0f) && lt < __builtin_inff());
    odd = static_cast<unsigned>(rows | (rows >> 32));
  };
  if (min(q0 + 1, W) < kSplitKeys)
    run(std::true_type{});
  else
    run(std::false_type{});
  // rows with finite scores and a non-finite o: again, key by key
  while (odd) {
    const int t = qw + __builtin_ctz(odd);
    odd &= odd - 1;
    exact_row<DH>(q_ + static_cast<size_t>(t) * x.q_stride, k_, v_, o_ + static_cast<size_t>(t) * ostride, x, c,
                  t, lane);
  }
}

namespace {

// With a workgroup a CU or fewer, each SIMD would have one wave, whose steps wait for each other: two share the
// keys then (17.5 us instead of 22 at B3 T1111 Hq6 Hkv2 dh128 W300, 7.3 instead of 8.1 at B1 T101 Hq4 dh64).
template <int DH> hipError_t launch(const AttnArgs &a, hipStream_t s) {
  constexpr unsigned kCus = 256;
  const long long groups = static_cast<long long>((a.T + kOwn - 1) / kOwn) * a.B * a.Hq;
  if (groups <= kCus && a.T > kBlk)
    attn_fwd<DH, 2><<<static_cast<unsigned>(groups), 64 * kWg * 2, 0, s>>>(a);
  else
    attn_fwd<DH, 1><<<dim3(grid_x(groups), grid_rows(groups)), 64 * kWg, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_local_attention(const AttnArgs &args, hipStream_t s) {
  AttnArgs a = args;
  a.window = std::min(a.window, a.T);
  a.sinks = std::min(a.sinks, a.T);
  switch (a.dh) {
    case 64: return launch<64>(a, s);
    case 128: return launch<128>(a, s);
    case 256: return launch<256>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace rglru
