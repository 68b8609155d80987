// rglru_linear.hip -- causal linear attention with a decay for each head (gfx950, bf16): prompts and single tokens.
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T  (dk x dv, fp32),   o_t = scale S_t^T q_t
// with g_t <= 0 a constant of the head or a value of each (token, head). For a chunk of 64 tokens with entering state
// S and b_t the sum of its g up to t:
//   o_t = scale (sum_{s <= t} exp(b_t - b_s) <q_t, k_s> v_s + exp(b_t) S^T q_t)
//   S'  = exp(b_63) S + sum_s exp(b_63 - b_s) k_s v_s^T
// All exponents are differences of one running sum taken before the exponential, so nothing is divided by a decay and
// strong decays only underflow. The sum is held in 64 bits and each difference is rounded once, so that the weights of
// tokens behind a strong decay are as exact as without it (in 32 bits, 48 decays of e^-103 in a chunk cost those behind
// them 2^-13). Tokens that forget the state are counted beside the sum: their decays may be infinite.
//
// linear_fwd: a workgroup walks the chunks of one (sequence, head, slice of up to 128 values, segment); each wave
// keeps S for 16 of the values (dk x 16 in accumulators). Per chunk, on 16x16x32 MFMAs:
//   P^T = K Q^T, its ten causal 16x16 tiles shared among the waves, decayed, and handed round in LDS as the next
//     product's operand;
//   O^T = S^T Q^T: S is the operand straight from its accumulators, as Q lies in their row order;
//   O^T += V^T P^T and S += K^T (w V), V and K read from LDS transposed, V once for both.
// S and P enter as bf16 hi + lo and w V as three bf16 terms (8 + 8 + 8 bits): the state is an fp32 result and o is
// then within the rounding of its own type; with one term each, o would be off by as much again for each of them.
//
// With few (sequence, head, slice)s the prompt is cut into segments: linear_state first forms the states of their own
// tokens (K and V only; of a segment whole, or of parts of it), and linear_fwd starts each segment from the chain of those
// before it: up to kFew states it forms the chain itself (at B8 T2048 H16 9.5 us of a launch less), else linear_carry has
// done so in place.
//
// Timed one call after another, all kernels: B8 T2048 H16 dk128 dv128 95 us, B1 T65536 H8 dk128 dv256 301 (607 MB, 110
// us at the 5.5 TB/s that reading a cache back reaches). In a trace, at lower clocks, B8 has 24 us of states and 87 of
// linear_fwd, B1 30, 9 of the chain and 351. A wave's chunk has 97 matrix instructions (59 without the lower terms) and
// some 530 vector ones (650 where two workgroups share a CU), 200 of them the splitting into terms. With one workgroup
// on each CU matrix units are busy for 27% of the time (B1: 33%), vector units for 39% (46%), LDS for 36%; two waves a
// SIMD hardly hide one behind the other, and the rest is waiting at the three barriers. With two workgroups a CU the
// waits overlap, but the states of twice the segments cost as much.
#include "rglru_attn.h"
#include "rglru_grid.h"
#include "rglru_launch.h"

#include <algorithm>

namespace rglru {

using namespace attn;

namespace {

constexpr int kC = 64;              // tokens per chunk
constexpr int kFew = 4;             // states that are chained where they are needed
constexpr float kLeast = -104.0f;   // exp of it is 0 in fp32: a smaller log decay (-inf) forgets the state
constexpr double kGone = -150.0;    // exp2 of it is 0 in fp32
constexpr double kLog2E = 1.4426950408889634;

// Inclusive running sum over the 64 lanes, in 64 bits.
template <int CTRL, int ROWS> __device__ __forceinline__ double plus_moved(double v) {
  const uint2 x = __builtin_bit_cast(uint2, v);
  const uint2 y = {static_cast<unsigned>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x.x), CTRL, ROWS, 0xF, false)),
                   static_cast<unsigned>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x.y), CTRL, ROWS, 0xF, false))};
  return v + __builtin_bit_cast(double, y);
}
__device__ __forceinline__ double wave_sum_up(double v) {
  v = plus_moved<0x111, 0xF>(v);  // row_shr:1
  v = plus_moved<0x112, 0xF>(v);  // row_shr:2
  v = plus_moved<0x114, 0xF>(v);  // row_shr:4
  v = plus_moved<0x118, 0xF>(v);  // row_shr:8
  v = plus_moved<0x142, 0xA>(v);  // row_bcast:15
  v = plus_moved<0x143, 0xC>(v);  // row_bcast:31
  return v;
}

// 8 fp32 values as bf16 terms: x = hi + mid (+ lo), each the rounding of what is left.
__device__ __forceinline__ u32x4_t split(float (&x)[8]) {
  u32x4_t h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    asm("" : "+v"(h[i]));  // (else the lower value is rounded a second time for the difference)
    x[2 * i] -= bf16lo(h[i]);
    x[2 * i + 1] -= bf16hi(h[i]);
  }
  return h;
}
__device__ __forceinline__ u32x4_t rounded(const float (&x)[8]) {
  u32x4_t h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  return h;
}

typedef __attribute__((address_space(3))) uint16_t lds_u16_t;
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef double f64x4_t __attribute__((ext_vector_type(4), aligned(16)));

// Whether any of 8 bf16 values is infinite or NaN: as integers without their sign, those are the largest.
__device__ __forceinline__ bool not_finite(u32x4_t v) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  u16x2_t top = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, v[i] & 0x7FFF7FFFu));
  return top[0] >= 0x7F80 || top[1] >= 0x7F80;
}

__device__ __forceinline__ f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

}  // namespace

// 64 rows of DH bf16 in LDS, 64 bytes apart beyond their length, the 16-byte chunk c of each 64 bytes of row r at c ^
// turn(r): what is read at once falls on different banks (16 rows at one chunk, 8 rows at 2 neighbouring chunks, 8 rows at
// one and the 8 others at its neighbour), and the steps along a row are constant offsets. Lanes are c = lane % 16, g = lane / 16.
template <int DH, int NT, bool ROOM> struct Rows64 {
  static constexpr unsigned kStride = 2 * DH + 64, kBytes = kC * kStride;
  static constexpr int kCPR = DH / 8, kN = kC * kCPR / NT;  // 16-byte chunks per row; per thread
  static constexpr int kRows = NT / kCPR;                   // rows that one of the threads' chunks covers
  // the chunks of rows `base` .. from memory, rows from `rows` on as zeros
  // (without ROOM the thread's terms are formed anew here and in put: kept through the walk, they take its registers)
  __device__ __forceinline__ static void load(u32x4_t (&x)[kN], const bf16_t *base, unsigned row_bytes, int rows, int tid) {
    if constexpr (!ROOM) asm volatile("" : "+v"(tid));
    const auto src = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<bf16_t *>(wave_uniform(base)), static_cast<short>(0),
        rows > 0 ? static_cast<int>(row_bytes * static_cast<unsigned>(min(rows, kC) - 1)) + DH * 2 : 0, kRawWord3);
    const unsigned at = static_cast<unsigned>(tid / kCPR) * row_bytes + (tid % kCPR) * 16;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      x[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(src, at + i * kRows * row_bytes, 0, 0));
  }
  __device__ __forceinline__ static int turn(int r) { return (2 * ((r >> 2) & 1)) ^ (3 * ((r >> 3) & 1)); }
  __device__ __forceinline__ static unsigned chunk(int r, int c) {  // of row r, its place
    return r * kStride + (c >> 2) * 64 + (((c & 3) ^ turn(r)) * 16);
  }
  // thread's chunk i is of row tid / kCPR + kRows i: its turn comes again after 16 rows
  static constexpr int kPar = kRows < 16 ? 16 / kRows : 1;
  __device__ __forceinline__ static void put(const u32x4_t (&x)[kN], unsigned lds, int tid) {
    if constexpr (!ROOM) asm volatile("" : "+v"(tid));
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int p = i % kPar;
      *(lds_u32x4_t *)static_cast<uintptr_t>(lds + chunk(tid / kCPR + kRows * p, tid % kCPR) + (i - p) * kRows * kStride) =
          x[i];
    }
  }
  // put with the order of two accumulators' rows in each 32 values: chunk g has 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3
  __device__ __forceinline__ static void put_paired(const u32x4_t (&x)[kN], unsigned lds, int tid) {
    if constexpr (!ROOM) asm volatile("" : "+v"(tid));
    const int r = tid / kCPR, c = tid % kCPR, to = (c & ~3) + 2 * (c & 1);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int p = i % kPar;
      const unsigned at = lds + (i - p) * kRows * kStride + 8 * ((c >> 1) & 1);
      *(lds_u32x2_t *)static_cast<uintptr_t>(at + chunk(r + kRows * p, to)) = u32x2_t{x[i][0], x[i][1]};
      *(lds_u32x2_t *)static_cast<uintptr_t>(at + chunk(r + kRows * p, to + 1)) = u32x2_t{x[i][2], x[i][3]};
    }
  }
  // operand, row c of the 16 at `lds`, k = what lies at values 32 st + 8 g ..
  __device__ __forceinline__ static unsigned row_lane(int lane) { return chunk(lane & 15, lane >> 4); }
  __device__ __forceinline__ static u32x4_t rows(unsigned lds, unsigned l, int st) {
    return *(lds_u32x4_t *)static_cast<uintptr_t>(l + lds + 64 * st);
  }
  // the same of rows as they came, k in the paired order
  struct PairLane {
    unsigned at[2];
  };
  __device__ __forceinline__ static PairLane pair_lane(int lane) {
    const int r = lane & 15, g = lane >> 4;
    return {{chunk(r, g >> 1) + 8 * (g & 1), chunk(r, 2 + (g >> 1)) + 8 * (g & 1)}};
  }
  __device__ __forceinline__ static u32x4_t pairs(unsigned lds, const PairLane &l, int st) {
    const u32x2_t a = *(lds_u32x2_t *)static_cast<uintptr_t>(l.at[0] + lds + 64 * st),
                  b = *(lds_u32x2_t *)static_cast<uintptr_t>(l.at[1] + lds + 64 * st);
    return u32x4_t{a[0], a[1], b[0], b[1]};
  }
  // operand, column 16 j + c, k = rows 32 st + 4 g .. and 32 st + 16 + 4 g ..: two accumulators' row order
  struct ColLane {
    unsigned at[2];
  };
  __device__ __forceinline__ static ColLane col_lane(int lane) {
    const int r = 4 * (lane >> 4) + ((lane & 15) >> 2), c = (lane & 3) >> 1;
    return {{chunk(r, c) + 8 * (lane & 1), chunk(r, 2 + c) + 8 * (lane & 1)}};
  }
  __device__ __forceinline__ static u32x4_t cols(unsigned lds, unsigned l, int st) {
    const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                  (lds_i16x4_t *)static_cast<uintptr_t>(l + lds + 32 * st * kStride)));
    const uint2 y = __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                   (lds_i16x4_t *)static_cast<uintptr_t>(l + lds + (32 * st + 16) * kStride)));
    return u32x4_t{x.x, x.y, y.x, y.y};
  }
  __device__ __forceinline__ static u32x4_t cols(unsigned lds, const ColLane &l, int st, int j) {
    return cols(lds + 64 * (j >> 1), l.at[j & 1], st);
  }
  // one value, for the few that are read alone
  __device__ __forceinline__ static float value(unsigned lds, int r, int d) {
    return bf16_to_f32(*(lds_u16_t *)static_cast<uintptr_t>(lds + chunk(r, d >> 3) + 2 * (d & 7)));
  }
};

// The decayed scores in LDS, as lanes read them: operand of (16 tokens j, 32 earlier ones p <= j / 2), hi then lo.
constexpr unsigned kScores = 6 * 64 * 16;
__device__ __forceinline__ constexpr unsigned scores_of(int j, int p) { return (j < 2 ? j : 2 * j - 2 + p) * 1024; }

// O^T += V^T P^T of each 16 tokens' own 32, one token at a time, in fp32. (The lane's terms are formed here: kept, they
// would take registers from the walk, which hardly ever comes here.)
template <typename VB> __device__ __forceinline__ void own_tokens(f32x4_t (&O)[4], unsigned ldv, unsigned ldp, int w, int lane) {
  asm volatile("" : "+v"(lane));
  const int c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    for (int s = 0; s < 16 * (1 + (j & 1)); ++s) {
      const unsigned at = ldp + scores_of(j, j >> 1) + (c + 16 * ((s >> 2) & 3)) * 16 + 8 * (s >> 4) + 2 * (s & 3);
      const float p = bf16_to_f32(*(lds_u16_t *)static_cast<uintptr_t>(at)) +
                      bf16_to_f32(*(lds_u16_t *)static_cast<uintptr_t>(at + kScores));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = p * VB::value(ldv, 32 * (j >> 1) + s, 16 * w + 4 * g + e);
        if (s <= 16 * (j & 1) + c) O[j][e] += x;
      }
    }
}

// 2^b, b rounded once: relatively off by 2^-24 |b| ln 2 and the exponential's own 2^-23, however large the sums that b is
// the difference of.
__device__ __forceinline__ float decay_of(double b) { return __builtin_amdgcn_exp2f(static_cast<float>(b)); }

// Of a chunk's tokens up to the lane's one, and of all: the summed log2 decays of those that do not forget the state, and
// the number of those that do.
struct Sums {
  double b, b_end;
  int f, f_end;
  // what is left of the lane's token after the chunk, with 2^later to come; of the state before it
  __device__ __forceinline__ float kept(double later) const { return f == f_end ? decay_of(b_end - b + later) : 0.0f; }
  __device__ __forceinline__ float before() const { return f == 0 ? decay_of(b) : 0.0f; }
};

// This workgroup's (sequence, head, slice, segment), and where its tokens are.
template <int DK, int DVS> struct Place {
  int b, seg, h, slice, len, t_lo, t_hi, t_end;
  size_t tok, head;
  const bf16_t *k, *v;
  const float *g;
  size_t g_stride;
  __device__ __forceinline__ bool find(const LinearArgs &a) {
    // Heads of one key head, and their slices, one after another: they read the same q and k. Workgroups go to the 8
    // dies (each with an L2 of its own) in turn, so each die takes one run of them.
    const int nsl = a.dv / DVS, per = a.H * nsl * a.run, eighth = per * a.B >> 3;
    int id = block_of(blockIdx.y);
    if (id < eighth * 8) id = (id & 7) * eighth + (id >> 3);
    b = uni(id / per);
    if (b >= a.B) return false;
    const int r0 = id - b * per;
    seg = uni(r0 / (a.H * nsl));
    const int r1 = r0 - seg * a.H * nsl;
    h = uni(r1 / nsl);
    slice = r1 - h * nsl;
    len = clamp_len(a.lens, b, a.T);
    t_lo = seg * a.seg_len;
    t_hi = t_lo + min(a.seg_len, a.T - t_lo);  // (t_lo + seg_len may pass 2^31)
    t_end = min(len, t_hi);
    tok = static_cast<size_t>(b) * a.T;
    head = static_cast<size_t>(b) * a.H + h;
    k = static_cast<const bf16_t *>(a.k) + tok * a.k_stride + static_cast<size_t>(key_head(a)) * DK;
    v = static_cast<const bf16_t *>(a.v) + tok * a.v_stride + static_cast<size_t>(h) * a.dv + slice * DVS;
    g = a.gated ? a.log_decay + tok * a.H + h : a.log_decay + h;
    g_stride = a.gated ? a.H : 0;
    return true;
  }
  __device__ __forceinline__ int key_head(const LinearArgs &a) const { return uni(h / (a.H / a.Hk)); }
  // log decay of token t + lane (behind the segment's last one: any)
  __device__ __forceinline__ float decay(int t, int lane) const {
    return g[static_cast<size_t>(min(t + lane, t_end - 1)) * g_stride];
  }
  // the running sums, from what decay() has loaded
  __device__ __forceinline__ Sums running(float x, int t, int lane) const {
    const bool live = t + lane < t_end, forgets = live && x < kLeast;
    const unsigned long long all = __ballot(forgets);
    Sums r;
    r.b = wave_sum_up(live && !forgets ? x * kLog2E : 0.0);
    r.f = __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(all >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(all), forgets));
    const uint2 last = __builtin_bit_cast(uint2, r.b);
    r.b_end = __builtin_bit_cast(double, uint2{static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(last.x), 63)),
                                               static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(last.y), 63))});
    r.f_end = __popcll(all);
    return r;
  }
};

// V's operand of 32 tokens, each times its weight, as three bf16 terms.
struct Weighted {
  u32x4_t hi, mid, lo;
};
__device__ __forceinline__ Weighted weighted(u32x4_t v, const float *w, int st, int g) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    x[e] = (e & 1 ? bf16hi(v[e >> 1]) : bf16lo(v[e >> 1])) * w[32 * st + 16 * (e >> 2) + 4 * g + (e & 3)];
  Weighted r;
  r.hi = split(x);
  r.mid = split(x);
  r.lo = rounded(x);
  return r;
}

// S += K^T (w V) of 64 tokens, four of S's tiles at a time.
template <int DK, typename KB> __device__ __forceinline__ void add_outer(f32x4_t (&S)[DK / 16], const u32x4_t (&v)[2],
                                                                         const float *w, unsigned ldk,
                                                                         const typename KB::ColLane &kl, int g) {
#pragma unroll
  for (int st = 0; st < 2; ++st) {
    const Weighted x = weighted(v[st], w, st, g);
#pragma unroll
    for (int n = 0; n < DK / 64; ++n) {
      f32x4_t *const s = S + 4 * n;
      u32x4_t kt[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) kt[i] = KB::cols(ldk, kl, st, 4 * n + i);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = mfma(kt[i], x.hi, s[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = mfma(kt[i], x.mid, s[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = mfma(kt[i], x.lo, s[i]);
    }
  }
}

// A wave's share of a state to memory and from it: dk = 16 i + 4 g + e of tile i, value c of the 16 from p on. (The
// lane's terms are formed here: kept from one call for the other, they take registers from the walk.)
template <int DK> __device__ __forceinline__ void store_state(const f32x4_t (&S)[DK / 16], float *p, int dv) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  float *const at = p + 4 * (lane >> 4) * dv + (lane & 15);
#pragma unroll
  for (int i = 0; i < DK / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) at[static_cast<size_t>(16 * i + e) * dv] = S[i][e];
}
template <int DK> __device__ __forceinline__ void load_state(f32x4_t (&S)[DK / 16], const float *p, int dv) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  const float *const at = p + 4 * (lane >> 4) * dv + (lane & 15);
#pragma unroll
  for (int i = 0; i < DK / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[i][e] = at[static_cast<size_t>(16 * i + e) * dv];
}

// Threads of a workgroup, a wave for 16 values. Registers: ROOM for one workgroup a CU, which keeps its addresses, or
// for two.
constexpr int threads_of(int DVS) { return DVS * 4; }
constexpr int waves_of(int DVS, bool ROOM) { return (ROOM ? 1 : 2) * (DVS / 64); }

// The state of the own tokens of a segment, or of a part of one, at its end (to the next one's a.seg), and its summed g (a.sums). Chunks from the
// last one back: once what follows has decayed by 2^-150 in all, which is 0 in fp32, no earlier token counts.
template <int DK, int DVS>
__global__ __launch_bounds__(threads_of(DVS), waves_of(DVS, DK == 256)) void linear_state(LinearArgs a) {
  constexpr int NT = threads_of(DVS);
  typedef Rows64<DK, NT, true> KB;
  typedef Rows64<DVS, NT, true> VB;
  __shared__ __attribute__((aligned(16))) unsigned char smem[KB::kBytes + VB::kBytes];
  __shared__ __attribute__((aligned(16))) float sw[DVS / 16][kC];  // each wave's own
  const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6), g = lane >> 4;
  const unsigned ldk = lds_addr(smem), ldv = ldk + KB::kBytes;
  Place<DK, DVS> at;
  if (!at.find(a)) return;
  const unsigned krb = static_cast<unsigned>(a.k_stride) * 2, vrb = static_cast<unsigned>(a.v_stride) * 2;
  f32x4_t S[DK / 16];
#pragma unroll
  for (int i = 0; i < DK / 16; ++i) S[i] = f32x4_t{};
  double later = 0.0;  // summed log2 decays of the chunks done
  u32x4_t kx[KB::kN], vx[VB::kN];
  float gx = 0.0f;
  auto load = [&](int t) {
    KB::load(kx, at.k + static_cast<size_t>(t) * a.k_stride, krb, at.t_end - t, tid);
    VB::load(vx, at.v + static_cast<size_t>(t) * a.v_stride, vrb, at.t_end - t, tid);
    gx = at.decay(t, lane);
  };
  const int n = at.t_end > at.t_lo ? (at.t_end - at.t_lo + kC - 1) / kC : 0;
  if (n) load(at.t_lo + (n - 1) * kC);
  const typename KB::ColLane kc = KB::col_lane(lane);
  const unsigned vc = ldv + 64 * (w >> 1) + (w & 1 ? VB::col_lane(lane).at[1] : VB::col_lane(lane).at[0]);
  for (int i = n - 1; i >= 0 && !(later <= kGone); --i) {
    KB::put(kx, ldk, tid);
    VB::put(vx, ldv, tid);
    const Sums sums = at.running(gx, at.t_lo + i * kC, lane);
    sw[w][lane] = sums.kept(later);
    later = sums.f_end ? kGone : later + sums.b_end;
    lds_barrier();
    if (i) load(at.t_lo + (i - 1) * kC);
    u32x4_t v[2];
#pragma unroll
    for (int st = 0; st < 2; ++st) v[st] = VB::cols(0, vc, st);
    add_outer<DK, KB>(S, v, sw[w], ldk, kc, g);
    lds_barrier();  // everyone is done with the chunk
  }
  if (tid == 0 && at.slice == 0) a.sums[at.head * a.states + at.seg] = static_cast<float>(later);
  store_state<DK>(S, a.seg + (at.head * (a.states + 1) + at.seg + 1) * static_cast<size_t>(DK) * a.dv + at.slice * DVS + 16 * w,
                  a.dv);
}

template <int DK, int DVS, bool ROOM>
__global__ __launch_bounds__(threads_of(DVS), waves_of(DVS, ROOM)) void linear_fwd(LinearArgs a) {
  constexpr int NW = DVS / 16, NT = threads_of(DVS);
  typedef Rows64<DK, NT, ROOM> KB;
  typedef Rows64<DVS, NT, ROOM> VB;
  __shared__ __attribute__((aligned(16))) unsigned char smem[2 * KB::kBytes + VB::kBytes + 2 * kScores];
  // b, the number that forget, scale exp(b), exp(b_63 - b); exp(b_63)
  __shared__ __attribute__((aligned(16))) double mb[kC];
  __shared__ __attribute__((aligned(16))) float me[kC], mw[kC];
  __shared__ __attribute__((aligned(16))) int mf[kC];
  __shared__ float mkeep;
  const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const unsigned ldk = lds_addr(smem), ldv = ldk + KB::kBytes, ldq = ldv + VB::kBytes, ldp = ldq + KB::kBytes;
  Place<DK, DVS> at;
  if (!at.find(a)) return;
  const bf16_t *const q_ = static_cast<const bf16_t *>(a.q) + at.tok * a.q_stride +
                           static_cast<size_t>(at.key_head(a)) * DK;
  const unsigned qrb = static_cast<unsigned>(a.q_stride) * 2, krb = static_cast<unsigned>(a.k_stride) * 2,
                 vrb = static_cast<unsigned>(a.v_stride) * 2;
  u32x4_t qx[KB::kN], kx[KB::kN], vx[VB::kN];
  float gx = 0.0f;  // (the last wave's)
  auto load = [&](int t) {
    KB::load(kx, at.k + static_cast<size_t>(t) * a.k_stride, krb, at.t_end - t, tid);
    if (w == NW - 1) gx = at.decay(t, lane);
  };
  auto load_qv = [&](int t) {
    KB::load(qx, q_ + static_cast<size_t>(t) * a.q_stride, qrb, at.t_end - t, tid);
    VB::load(vx, at.v + static_cast<size_t>(t) * a.v_stride, vrb, at.t_end - t, tid);
  };
  f32x4_t S[DK / 16];
  const size_t dkv = static_cast<size_t>(DK) * a.dv;
  const int col = at.slice * DVS + 16 * w;
  const int before = at.seg * a.sub;  // states before the segment
  if (const float *from = a.chained ? a.seg + (at.head * (a.states + 1) + before) * dkv : a.s0 ? a.s0 + at.head * dkv : nullptr) {
    load_state<DK>(S, from + col, a.dv);
  } else {
#pragma unroll
    for (int i = 0; i < DK / 16; ++i) S[i] = f32x4_t{};
  }
  for (int j = 0; !a.chained && j < before; ++j) {
    const float keep = __builtin_amdgcn_exp2f(uniform_load(a.sums, at.head * a.states + j));
    f32x4_t own[DK / 16];
    load_state<DK>(own, a.seg + (at.head * (a.states + 1) + j + 1) * dkv + col, a.dv);
#pragma unroll
    for (int i = 0; i < DK / 16; ++i) S[i] = S[i] * keep + own[i];
  }
  if (at.t_lo < at.t_end) {
    load(at.t_lo);
    load_qv(at.t_lo);
  }
  bf16_t *const o_ = static_cast<bf16_t *>(a.o) + (at.tok * a.H + at.h) * a.dv + col;
  const size_t o_stride = static_cast<size_t>(a.H) * a.dv;
  const typename KB::ColLane kc = KB::col_lane(lane);
  const typename KB::PairLane kr = KB::pair_lane(lane);
  const unsigned vc = ldv + 64 * (w >> 1) + (w & 1 ? VB::col_lane(lane).at[1] : VB::col_lane(lane).at[0]);
  const unsigned qr = ldq + KB::row_lane(lane), pl = ldp + lane * 16;
  if (w == 0) {  // of the scores' operands, the tokens behind the 16 of an even j: never written again
#pragma unroll
    for (int j = 0; j < 4; j += 2)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        *(lds_u32x2_t *)static_cast<uintptr_t>(pl + scores_of(j, j >> 1) + 8 + x * kScores) = u32x2_t{};
  }

  // o of a chunk goes to memory through q's place, in whole rows, where the two have rows of one length (each thread's
  // 16 bytes, before its wave puts the next q there)
  constexpr bool kThrough = DK == DVS;
  auto store_rows = [&](int t0) {
    int x = tid;
    if constexpr (!ROOM) asm volatile("" : "+v"(x));
#pragma unroll
    for (int i = 0; i < VB::kN; ++i) {
      const int r = x / VB::kCPR + VB::kRows * i, row = t0 + r;
      u32x4_t y = *(lds_u32x4_t *)static_cast<uintptr_t>(ldq + VB::chunk(r, x % VB::kCPR));
      if (row >= at.len) y = u32x4_t{};
      if (row < at.t_hi) *reinterpret_cast<u32x4_t *>(o_ - 16 * w + row * o_stride + 8 * (x % VB::kCPR)) = y;
    }
  };
  for (int t = at.t_lo; t < at.t_end; t += kC) {
    KB::put(kx, ldk, tid);
    if (kThrough && t > at.t_lo) store_rows(t - kC);
    KB::put_paired(qx, ldq, tid);
    VB::put(vx, ldv, tid);
    if (w == NW - 1) {  // (the first ones have two tiles of scores)
      const Sums sums = at.running(gx, t, lane);
      mb[lane] = sums.b;
      mf[lane] = sums.f;
      me[lane] = sums.before() * a.scale;
      mw[lane] = sums.kept(0.0);
      if (lane == 63) mkeep = sums.before();
    }
    lds_barrier();
    if (t + kC < at.t_end) load(t + kC);
    // ---- O^T = S^T Q^T, rows scaled by scale exp(b_t): value 16 w + 4 g + e, token 16 j + c
    f32x4_t O[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) O[j] = f32x4_t{};
#pragma unroll
    for (int n = 0; n < DK / 32; ++n) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = S[2 * n + (e >> 2)][e & 3];
      const u32x4_t hi = split(f), lo = rounded(f);
      u32x4_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = KB::rows(16 * j * KB::kStride, qr, n);
#pragma unroll
      for (int j = 0; j < 4; ++j) O[j] = mfma(hi, q[j], O[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) O[j] = mfma(lo, q[j], O[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) O[j] *= me[16 * j + c];
    // ---- P^T: tile of tokens 16 j .. against 16 i ..
    for (int n = w; n < 10; n += NW) {
      const int j = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3, i = n - j * (j + 1) / 2;
      f32x4_t p = f32x4_t{};
      const unsigned k0 = ldk + 16 * i * KB::kStride, q0 = qr + 16 * j * KB::kStride;
#pragma unroll
      for (int d = 0; d < DK / 32; ++d) p = mfma(KB::pairs(k0, kr, d), KB::rows(0, q0, d), p);
      const double btt = mb[16 * j + c];
      const int ftt = mf[16 * j + c];
      const f64x4_t bs = *reinterpret_cast<const f64x4_t *>(&mb[16 * i + 4 * g]);
      const i32x4_t fs = *reinterpret_cast<const i32x4_t *>(&mf[16 * i + 4 * g]);
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = p[e] * a.scale * decay_of(btt - bs[e]);
        x[e] = (i < j || 4 * g + e <= c) && fs[e] == ftt ? f : 0.0f;
      }
      const u32x2_t hi = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
      const u32x2_t lo = {pack_bf16x2(x[0] - bf16lo(hi[0]), x[1] - bf16hi(hi[0])),
                          pack_bf16x2(x[2] - bf16lo(hi[1]), x[3] - bf16hi(hi[1]))};
      const unsigned to = pl + scores_of(j, i >> 1) + 8 * (i & 1);
      *(lds_u32x2_t *)static_cast<uintptr_t>(to) = hi;
      *(lds_u32x2_t *)static_cast<uintptr_t>(to + kScores) = lo;
    }
    u32x4_t v[2];
#pragma unroll
    for (int st = 0; st < 2; ++st) v[st] = VB::cols(0, vc, st);
    // (not with the keys: registers would be spilled, and a spilled load is waited for)
    if (t + kC < at.t_end) load_qv(t + kC);
    lds_barrier();  // the scores are there
    // ---- O^T += V^T P^T. Where a v is infinite or NaN, 0 times it is not 0: each token's own 32 are left out here
    // and go one by one
    const bool odd = __any(not_finite(v[0]) || not_finite(v[1]));
    const unsigned own = odd ? 0u : ~0u;
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int j = 2 * st; j < 4; ++j) {
        const unsigned from = pl + scores_of(j, st);
        const u32x4_t x = st == j >> 1 ? v[st] & own : v[st];
        O[j] = mfma(x, *(lds_u32x4_t *)static_cast<uintptr_t>(from), O[j]);
        O[j] = mfma(x, *(lds_u32x4_t *)static_cast<uintptr_t>(from + kScores), O[j]);
      }
    if (odd) own_tokens<VB>(O, ldv, ldp, w, lane);
    int cr = c;
    if constexpr (!ROOM) asm volatile("" : "+v"(cr));  // (addresses of rows formed here, as above)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = t + 16 * j + cr;
      u32x2_t x = {pack_bf16x2(O[j][0], O[j][1]), pack_bf16x2(O[j][2], O[j][3])};
      if constexpr (kThrough) {
        *(lds_u32x2_t *)static_cast<uintptr_t>(ldq + VB::chunk(16 * j + cr, 2 * w + (g >> 1)) + 8 * (g & 1)) = x;
      } else {
        if (row >= at.len) x = u32x2_t{};
        if (row < at.t_hi) *reinterpret_cast<u32x2_t *>(o_ + row * o_stride + 4 * g) = x;
      }
    }
    // ---- S decays, and takes the chunk's tokens
    const float keep = mkeep;
#pragma unroll
    for (int i = 0; i < DK / 16; ++i) S[i] *= keep;
    add_outer<DK, KB>(S, v, mw, ldk, kc, g);
    lds_barrier();  // everyone is done with the chunk
  }
  // rows behind the sequence, from the first whole chunk on
  const int z0 = at.t_lo < at.t_end ? at.t_lo + (at.t_end - at.t_lo + kC - 1) / kC * kC : at.t_lo;
  if (kThrough && z0 > at.t_lo) store_rows(z0 - kC);
  for (long long i = z0 * 2LL + lane; i < at.t_hi * 2LL; i += 64)
    *reinterpret_cast<u32x4_t *>(o_ + static_cast<size_t>(i >> 1) * o_stride + 8 * static_cast<int>(i & 1)) = u32x4_t{};
  if (!a.s_out || at.seg != a.segs - 1) return;
  store_state<DK>(S, a.s_out + at.head * dkv + col, a.dv);
}

// Segments' own states to the states they end with, S_j = exp(sum of g) S_{j-1} + own, in place; the first one's from
// s0. 4 values a thread.
__global__ __launch_bounds__(256) void linear_carry(LinearArgs a) {
  const size_t dkv = static_cast<size_t>(a.dk) * a.dv, quads = dkv / 4;
  const size_t i = static_cast<size_t>(block_of(blockIdx.y)) * 256 + threadIdx.x;
  const size_t head = i / quads;
  if (head >= static_cast<size_t>(a.B) * a.H) return;
  const size_t at = (i - head * quads) * 4;
  f32x4_t s = a.s0 ? *reinterpret_cast<const f32x4_t *>(a.s0 + head * dkv + at) : f32x4_t{};
  const int n = a.states;
  float *const own = a.seg + head * (n + 1) * dkv + at;
  *reinterpret_cast<f32x4_t *>(own) = s;
  constexpr int kFly = 4;
  for (int j0 = 0; j0 < n; j0 += kFly) {
    f32x4_t u[kFly];
#pragma unroll
    for (int j = 0; j < kFly; ++j)
      if (j0 + j < n) u[j] = *reinterpret_cast<const f32x4_t *>(own + (j0 + j + 1) * dkv);
#pragma unroll
    for (int j = 0; j < kFly; ++j)
      if (j0 + j < n) {
        const float keep = __builtin_amdgcn_exp2f(a.sums[head * n + j0 + j]);
        s = s * keep + u[j];
        *reinterpret_cast<f32x4_t *>(own + (j0 + j + 1) * dkv) = s;
      }
  }
}

// One token: workgroup = (sequence, head, COLS of the values), the state read and written once. A row of the slice
// is COLS / 4 lanes' 16 bytes; rows are dealt to the lane groups, whose shares of o meet in LDS. Bound by memory: 4096
// states of dk128 dv256 in 210 us (1.07 GB, 5.1 TB/s; a plain copy of 1 GiB 5.2), 8 of dk128 dv128 in 3.4 us.
template <int COLS> __global__ __launch_bounds__(256) void linear_step(LinearStepArgs a) {
  constexpr int kLanes = COLS / 4, kGroups = 256 / kLanes, kFly = 8;
  __shared__ float qs[256], ks[256];
  __shared__ __attribute__((aligned(16))) float part[kGroups][COLS];
  const int nsl = a.dv / COLS, id = block_of(blockIdx.y), row = id / nsl, slice = id - row * nsl;
  if (row >= a.N * a.H) return;
  const int n = row / a.H, h = row - n * a.H, kh = h / (a.H / a.Hk);
  const int tid = threadIdx.x, c = tid % kLanes, grp = tid / kLanes;
  const bf16_t *const q = static_cast<const bf16_t *>(a.q) + n * a.q_stride + static_cast<size_t>(kh) * a.dk;
  const bf16_t *const k = static_cast<const bf16_t *>(a.k) + n * a.k_stride + static_cast<size_t>(kh) * a.dk;
  const int at = slice * COLS + 4 * c;
  const size_t base = static_cast<size_t>(row) * a.dk * a.dv + at;
  const float *const in = a.s_in + base;
  float *const out = a.s_out + base;
  f32x4_t s[kFly];
  auto load = [&](int r) {
#pragma unroll
    for (int j = 0; j < kFly; ++j)
      if (r + j * kGroups < a.dk) s[j] = *reinterpret_cast<const f32x4_t *>(in + static_cast<size_t>(r + j * kGroups) * a.dv);
  };
  load(grp);
  if (tid < a.dk) {
    qs[tid] = bf16_to_f32(q[tid]) * a.scale;
    ks[tid] = bf16_to_f32(k[tid]);
  }
  const float g = a.log_decay[a.gated ? row : h];
  const float keep = g < kLeast ? 0.0f : __builtin_amdgcn_exp2f(g * kLn2Inv);
  const u32x2_t vw = *reinterpret_cast<const u32x2_t *>(static_cast<const bf16_t *>(a.v) + n * a.v_stride +
                                                        static_cast<size_t>(h) * a.dv + at);
  const f32x4_t v = {bf16lo(vw[0]), bf16hi(vw[0]), bf16lo(vw[1]), bf16hi(vw[1])};
  __syncthreads();
  f32x4_t o = {};
  for (int r = grp; r < a.dk; r += kFly * kGroups) {
    if (r != grp) load(r);
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      const int rr = r + j * kGroups;
      if (rr < a.dk) {
        const f32x4_t x = s[j] * keep + v * ks[rr];
        *reinterpret_cast<f32x4_t *>(out + static_cast<size_t>(rr) * a.dv) = x;
        o += x * qs[rr];
      }
    }
  }
  *reinterpret_cast<f32x4_t *>(&part[grp][4 * c]) = o;
  __syncthreads();
  if (tid < COLS) {
    float x = 0.0f;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) x += part[j][tid];
    static_cast<bf16_t *>(a.o)[static_cast<size_t>(row) * a.dv + slice * COLS + tid] = f32_to_bf16(x);
  }
}

// Segments of a prompt: 256 workgroups, one a CU, where a workgroup's state has 16384 values or more (more segments are
// more states to form: B1 T32768 H16 dk256 dv256 492 us, with 512 workgroups 550; B8 T2048 H16 dk128 dv128 95 and 107), else
// 512 (B6 T4096 H16 dk64 dv128 109 us, with 256 128); 320 leave some CUs twice the others' work (728, 95, 140). Of two chunks
// at least (B1 T2048 H8 dk128 dv128 30 us, with four 36, with one 34.5; T128 11.5, with one 15).
LinearPlan linear_plan(int B, int T, int H, int dk, int dv) {
  const int dvs = dv == 64 ? 64 : 128;
  const long long groups = static_cast<long long>(B) * H * (dv / dvs);
  const int chunks = (T + kC - 1) / kC;
  const int target = dk * dvs < 16384 ? 512 : 256;
  long long segs = std::max<long long>(target / groups, 1);
  segs = std::min<long long>(segs, std::max(chunks / 2, 1));
  const int in_seg = static_cast<int>((chunks + segs - 1) / segs);
  LinearPlan p;
  // the states of few segments in parts, where forming them leaves CUs idle and the chain of them stays short (B8 T2048
  // H16 dk128 dv128: 95 us, whole 103; B16 T1024 H8 dk256 dv128 88 and 91; but B1 T2048 H8 dk128 dv128 with 30 states 37,
  // with 15 30)
  const long long before = std::max((chunks + in_seg - 1) / in_seg - 1, 1);
  const int sub = static_cast<int>(std::max<long long>(
      std::min<long long>({target / (before * groups), kFew / before, in_seg}), 1));
  const int in_state = (in_seg + sub - 1) / sub;
  p.sub = (in_seg + in_state - 1) / in_state;
  p.seg_len = p.sub * in_state * kC;
  p.segs = static_cast<int>((static_cast<long long>(T) + p.seg_len - 1) / p.seg_len);  // (T alone may be near 2^31)
  p.states = (p.segs - 1) * p.sub;
  return p;
}

namespace {

template <int DK, int DVS> hipError_t launch(LinearArgs a, hipStream_t s) {
  const long long rows = static_cast<long long>(a.B) * a.H * (a.dv / DVS);
  if (a.states) {
    const int seg_len = a.seg_len;
    a.run = a.states;
    a.seg_len /= a.sub;
    const long long g = rows * a.run;
    linear_state<DK, DVS><<<dim3(grid_x(g), grid_rows(g)), threads_of(DVS), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // (where the last state goes over the first one, the segments need a copy of that)
    a.chained = a.states > kFew || (a.s0 && a.s_out == a.s0);
    a.seg_len = seg_len;
  }
  if (a.chained) {
    const long long c = (static_cast<long long>(a.B) * a.H * DK * (a.dv / 4) + 255) / 256;
    linear_carry<<<dim3(grid_x(c), grid_rows(c)), 256, 0, s>>>(a);
    const hipError_t f = hipGetLastError();
    if (f != hipSuccess) return f;
  }
  a.run = a.segs;
  const long long g = rows * a.run;
  // dk128 dv128: room for two workgroups a CU where there are more than 256 (B24 T2048 H16, 384: 245 us, with
  // room for one 267; B32 T1024, 512: 148 and 158; but B8 T2048, 256: 101 and 95). Smaller states leave it anyway, larger ones never.
  const bool room = DK * DVS > 16384 || (DK * DVS == 16384 && (DK == 256 || g <= 256));
  const dim3 grid(grid_x(g), grid_rows(g));
  if constexpr (DK * DVS >= 16384)
    if (room) {
      linear_fwd<DK, DVS, true><<<grid, threads_of(DVS), 0, s>>>(a);
      return hipGetLastError();
    }
  if constexpr (DK < 256) linear_fwd<DK, DVS, false><<<grid, threads_of(DVS), 0, s>>>(a);
  return hipGetLastError();
}

template <int COLS> hipError_t launch(const LinearStepArgs &a, hipStream_t s) {
  const long long g = static_cast<long long>(a.N) * a.H * (a.dv / COLS);
  linear_step<COLS><<<dim3(grid_x(g), grid_rows(g)), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_attention(const LinearArgs &a, hipStream_t s) {
  switch (a.dk) {
    case 64: return a.dv == 64 ? launch<64, 64>(a, s) : launch<64, 128>(a, s);
    case 128: return a.dv == 64 ? launch<128, 64>(a, s) : launch<128, 128>(a, s);
    case 256: return a.dv == 64 ? launch<256, 64>(a, s) : launch<256, 128>(a, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_linear_step(const LinearStepArgs &a, hipStream_t s) {
  // 64 values for a workgroup (dk128 dv256, 4096 rows: 210 us, with 128 values 218, with 256 233, with 32 224); 32 while
  // that leaves the chip short of workgroups, the sooner the longer each one is (dk128 dv128: 16 rows 3.1 us, with 64
  // values 3.4, 512 rows 13.4 and 11.4; dk256 dv256: 32 rows 5.2 and 7.9, 512 rows 42 and 41)
  const long long groups = static_cast<long long>(a.N) * a.H * (a.dv / 64);
  return groups <= 2 * a.dk ? launch<32>(a, s) : launch<64>(a, s);
}

}  // namespace rglru
