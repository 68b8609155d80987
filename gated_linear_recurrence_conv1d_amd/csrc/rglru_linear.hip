// rglru_linear.hip -- causal linear attention with a decay for each head (gfx950, bf16): prompts and single tokens.
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T  (dk x dv, fp32),   o_t = scale S_t^T q_t
// with g_t <= 0 a constant of the head or a value of each (token, head). For a chunk of 64 tokens with entering state
// S and b_t the sum of its g up to t:
//   o_t = scale (sum_{s <= t} exp(b_t - b_s) <q_t, k_s> v_s + exp(b_t) S^T q_t)
//   S'  = exp(b_63) S + sum_s exp(b_63 - b_s) k_s v_s^T
// All exponents are differences of one running sum taken before the exponential, so nothing is divided by a decay and
// strong decays only underflow.
//
// linear_fwd: a workgroup walks the chunks of one (sequence, head, slice of up to 128 values, segment); each wave
// keeps S for 32 of the values (dk x 32 in accumulators). Per chunk, on 32x32x16 MFMAs:
//   P^T = K Q^T, its three causal 32x32 tiles shared among the waves, decayed, and handed round in LDS as the next
//     product's operand;
//   O^T = S^T Q^T: S is the operand straight from its accumulators, as Q takes its k index in their row order;
//   O^T += V^T P^T and S += K^T (w V), V and K read from LDS transposed, V once for both.
// S and P enter as bf16 hi + lo and w V as three bf16 terms (8 + 8 + 8 bits): the state is an fp32 result and o is
// then within the rounding of its own type; with one term each, o would be off by as much again for each of them.
//
// With few (sequence, head, slice)s the prompt is cut into segments: linear_fwd<.., STATE> first forms each
// segment's own state (K and V only), linear_carry chains them (from a copy of the first state: the last one may go
// where that is), and linear_fwd starts each segment from its state.
#include "rglru_attn.h"
#include "rglru_grid.h"
#include "rglru_launch.h"

#include <algorithm>

namespace rglru {

using namespace attn;

namespace {

constexpr int kC = 64;              // tokens per chunk
constexpr float kLeast = -104.0f;   // exp of it is 0 in fp32: a smaller log decay (-inf: forget) counts as this

// Inclusive running sum over the 64 lanes.
__device__ __forceinline__ float wave_sum_up(float v) {
  auto add = [](float x, int y) { return x + __int_as_float(y); };
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x111, 0xF, 0xF, false));  // row_shr:1
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x112, 0xF, 0xF, false));  // row_shr:2
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x114, 0xF, 0xF, false));  // row_shr:4
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x118, 0xF, 0xF, false));  // row_shr:8
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xA, 0xF, false));  // row_bcast:15
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xC, 0xF, false));  // row_bcast:31
  return v;
}

__device__ __forceinline__ float log2_decay(float g) { return (g < kLeast ? kLeast : g) * kLn2Inv; }

// 8 fp32 values as bf16 terms: x = hi + mid (+ lo), each the rounding of what is left.
__device__ __forceinline__ u32x4_t split(float (&x)[8]) {
  u32x4_t h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    x[2 * i] -= bf16lo(h[i]);
    x[2 * i + 1] -= bf16hi(h[i]);
  }
  return h;
}

typedef __attribute__((address_space(3))) uint16_t lds_u16_t;

// Whether any of 8 bf16 values is infinite or NaN: as integers without their sign, those are the largest.
__device__ __forceinline__ bool not_finite(u32x4_t v) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  u16x2_t top = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, v[i] & 0x7FFF7FFFu));
  return top[0] >= 0x7F80 || top[1] >= 0x7F80;
}

__device__ __forceinline__ f32x16_t mfma(u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

}  // namespace

// STATE: only the state at the segment's end from a zero one (into the next one's a.seg), and the segment's summed g (a.sums).
template <int DK, int DVS, bool STATE>
__global__ __launch_bounds__(DVS * 2, DK == 256 ? 1 : 2) void linear_fwd(LinearArgs a) {
  constexpr int NW = DVS / 32;
  typedef Blk<DK, NW> KB;
  typedef Blk<DVS, NW> VB;
  constexpr int kQB = 2 * KB::kBytes, kVB = 2 * VB::kBytes;  // 64 rows
  // the product's operands as lanes read them: [tile][step][lane], tiles (t0, s0), (t1, s0), (t1, s1), hi then lo
  constexpr int kPB = 3 * 2 * 64 * 16;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[(STATE ? 1 : 2) * kQB + kVB + (STATE ? 0 : 2 * kPB)];
  __shared__ __attribute__((aligned(16))) float sb[NW][3][kC];  // each wave's own: b, scale exp(b), exp(b_63 - b)
  const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6);
  const int lrow = lane & 31, half = lane >> 5;
  const unsigned ldk = lds_addr(smem), ldv = ldk + kQB, ldq = ldv + kVB, ldp = ldq + kQB;
  const int id = block_of(blockIdx.y);
  const int nsl = a.dv / DVS, per = a.H * nsl * a.run;
  // (heads of one key head, and their slices, one after another: they read the same q and k)
  const int b = uni(id / per);
  if (b >= a.B) return;
  const int r0 = id - b * per, seg = uni(r0 / (a.H * nsl)), r1 = r0 - seg * a.H * nsl;
  const int h = uni(r1 / nsl), slice = r1 - h * nsl;
  const int kh = uni(h / (a.H / a.Hk));
  const int T = a.T, len = clamp_len(a.lens, b, T);
  const int t_lo = seg * a.seg_len, t_hi = min(T, t_lo + a.seg_len), t_end = min(len, t_hi);
  const size_t tok = static_cast<size_t>(b) * T;
  const bf16_t *const q_ = static_cast<const bf16_t *>(a.q) + tok * a.q_stride + static_cast<size_t>(kh) * DK;
  const bf16_t *const k_ = static_cast<const bf16_t *>(a.k) + tok * a.k_stride + static_cast<size_t>(kh) * DK;
  const bf16_t *const v_ = static_cast<const bf16_t *>(a.v) + tok * a.v_stride + static_cast<size_t>(h) * a.dv +
                           slice * DVS;
  const float *const g_ = a.gated ? a.log_decay + tok * a.H + h : a.log_decay + h;
  const size_t g_stride = a.gated ? a.H : 0;
  const unsigned qrb = static_cast<unsigned>(a.q_stride) * 2, krb = static_cast<unsigned>(a.k_stride) * 2,
                 vrb = static_cast<unsigned>(a.v_stride) * 2;
  const typename KB::Lane ql = KB::load_lane(w, lane, qrb), kl = KB::load_lane(w, lane, krb);
  const typename VB::Lane vl = VB::load_lane(w, lane, vrb);

  // the state, dk = 32 i + 8 (e / 4) + 4 half + e % 4 of tile i, value 32 w + lane % 32 of the slice
  f32x16_t S[DK / 32];
  const size_t head = static_cast<size_t>(b) * a.H + h, dkv = static_cast<size_t>(DK) * a.dv;
  const int col = slice * DVS + 32 * w + lrow;
  {
    const float *from = STATE ? nullptr : a.segs == 1 ? a.s0 : a.seg;
    if (from) from += (head * a.segs + seg) * dkv + col;
#pragma unroll
    for (int i = 0; i < DK / 32; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        S[i][e] = from ? from[static_cast<size_t>(32 * i + 8 * (e >> 2) + 4 * half + (e & 3)) * a.dv] : 0.0f;
  }
  float total = 0.0f;
  const unsigned krow = KB::row_lane(lane), kcol = KB::col_lane(lane), vcol = VB::col_lane(lane);
  bf16_t *const o_ = static_cast<bf16_t *>(a.o) + (tok * a.H + h) * a.dv + slice * DVS + 32 * w;
  const size_t o_stride = static_cast<size_t>(a.H) * a.dv;
  float *const mb = sb[w][0], *const me = sb[w][1], *const mw = sb[w][2];

  auto load_chunk = [&](int t) {
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {  // 32 rows each; rows from len on read zero
      const int u = t + 32 * hb, rows = len - u;
      const size_t at = rows > 0 ? u : 0;
      const auto sk = KB::rsrc(k_ + at * a.k_stride, krb, rows), sv = VB::rsrc(v_ + at * a.v_stride, vrb, rows);
#pragma unroll
      for (int i = 0; i < KB::kLPW; ++i) KB::load(sk, krb, i, w, kl, ldk + hb * KB::kBytes);
#pragma unroll
      for (int i = 0; i < VB::kLPW; ++i) VB::load(sv, vrb, i, w, vl, ldv + hb * VB::kBytes);
      if constexpr (!STATE) {
        const auto sq = KB::rsrc(q_ + at * a.q_stride, qrb, rows);
#pragma unroll
        for (int i = 0; i < KB::kLPW; ++i) KB::load(sq, qrb, i, w, ql, ldq + hb * KB::kBytes);
      }
    }
  };
  auto load_decay = [&](int t) { return t + lane < t_end ? log2_decay(g_[static_cast<size_t>(t + lane) * g_stride]) : 0.0f; };

  if (t_lo < t_end) load_chunk(t_lo);
  float g_next = t_lo < t_end ? load_decay(t_lo) : 0.0f;
  for (int t = t_lo; t < t_end; t += kC) {
    // ---- the chunk's running sum of log2 decays, each wave for itself
    const float bt = wave_sum_up(g_next);
    const float b_end = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bt), 63));
    mb[lane] = bt;
    me[lane] = __builtin_amdgcn_exp2f(bt) * a.scale;
    mw[lane] = __builtin_amdgcn_exp2f(b_end - bt);
    if constexpr (STATE) total += b_end;
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's rows landed
    lds_barrier();
    g_next = t + kC < t_end ? load_decay(t + kC) : 0.0f;
    f32x16_t O[2];  // O^T: value 32 w + 8 (e / 4) + 4 half + e % 4 of the slice, token 32 tile + lane % 32
    if constexpr (!STATE) {
      // ---- P^T
      for (int tile = w; tile < 3; tile += NW) {
        const int tt = tile > 0 ? 1 : 0, ss = tile > 1 ? 1 : 0;
        f32x16_t p = f32x16_t{};
        unsigned ka = ldk + ss * KB::kBytes + krow, qa = ldq + tt * KB::kBytes + krow;
        asm volatile("" : "+v"(ka), "+v"(qa));
#pragma unroll
        for (int d = 0; d < KB::kKS; ++d)
          p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(KB::rows(ka, d), KB::rows(qa, d), p, 0, 0, 0);
        const float btt = mb[32 * tt + lrow];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int s = 16 * st + 8 * (e >> 2) + 4 * half + (e & 3);
            const float f = p[8 * st + e] * a.scale * __builtin_amdgcn_exp2f(btt - mb[32 * ss + s]);
            x[e] = tt > ss || s <= lrow ? f : 0.0f;
          }
          const unsigned at = ldp + ((tile * 2 + st) * 64 + lane) * 16;
          *(lds_u32x4_t *)static_cast<uintptr_t>(at) = split(x);
          *(lds_u32x4_t *)static_cast<uintptr_t>(at + kPB) = split(x);
        }
      }
      lds_barrier();
      // ---- O^T = S^T Q^T, rows scaled by scale exp(b_t)
      O[0] = O[1] = f32x16_t{};
      unsigned qa[2][2];  // row 32 tile + lane % 32: its chunk for values 4 half .. of 8 and of the next 8
      const int rq = lane & 31;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          qa[tt][x] = ldq + tt * KB::kBytes + rq * KB::kRowBytes + ((x ^ KB::swz(rq)) * 16) + 8 * half;
          asm volatile("" : "+v"(qa[tt][x]));
        }
#pragma unroll
      for (int i = 0; i < DK / 32; ++i)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = S[i][8 * st + e];
          const u32x4_t hi = split(x), lo = split(x);
#pragma unroll
          for (int tt = 0; tt < 2; ++tt) {
            const unsigned step = 32u * (2 * i + st);
            const u32x2_t q0 = *(lds_u32x2_t *)static_cast<uintptr_t>(qa[tt][0] ^ step),
                          q1 = *(lds_u32x2_t *)static_cast<uintptr_t>(qa[tt][1] ^ step);
            const u32x4_t qv = {q0[0], q0[1], q1[0], q1[1]};
            O[tt] = mfma(hi, qv, O[tt]);
            O[tt] = mfma(lo, qv, O[tt]);
          }
        }
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) O[tt] *= me[32 * tt + lrow];
    }
    // ---- S decays; then O^T += V^T P^T and S += K^T (w V), 16 tokens at a time
    const float keep = __builtin_amdgcn_exp2f(b_end);
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) S[i] *= keep;
    unsigned va = ldv + vcol, ka = ldk + kcol;
    asm volatile("" : "+v"(va), "+v"(ka));
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      const u32x4_t v = __builtin_bit_cast(u32x4_t, VB::cols(va, st, w));
      if constexpr (!STATE) {
        // a token's own tile: 0 * v is not 0 where a later token's v is infinite or NaN, those go one by one
        const bool odd = __any(not_finite(v));
#pragma unroll
        for (int tt = st >> 1; tt < 2; ++tt) {
          const unsigned at = ldp + (((tt + (st >> 1)) * 2 + (st & 1)) * 64 + lane) * 16;
          if (tt == st >> 1 && odd) {
            const unsigned vrows = ldv + tt * VB::kBytes, prow = ldp + ((2 * tt * 2 + (st & 1)) * 64 + lrow) * 16;
            for (int s = 0; s < 16; ++s) {
              const unsigned pa = prow + ((s >> 2) & 1) * 512 + ((s & 3) + 4 * (s >> 3)) * 2;
              const float p = bf16_to_f32(*(lds_u16_t *)static_cast<uintptr_t>(pa)) +
                              bf16_to_f32(*(lds_u16_t *)static_cast<uintptr_t>(pa + kPB));
              const int row = 16 * (st & 1) + s;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int d = 32 * w + 8 * (e >> 2) + 4 * half + (e & 3);
                const unsigned va1 = vrows + row * VB::kRowBytes + (((d >> 3) ^ VB::swz(row)) * 16) + (d & 7) * 2;
                const float x = p * bf16_to_f32(*(lds_u16_t *)static_cast<uintptr_t>(va1));
                if (row <= lrow) O[tt][e] += x;
              }
            }
            continue;
          }
          O[tt] = mfma(v, *(lds_u32x4_t *)static_cast<uintptr_t>(at), O[tt]);
          O[tt] = mfma(v, *(lds_u32x4_t *)static_cast<uintptr_t>(at + kPB), O[tt]);
        }
      }
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = (e & 1 ? bf16hi(v[e >> 1]) : bf16lo(v[e >> 1])) * mw[16 * st + 8 * (e >> 2) + 4 * half + (e & 3)];
      const u32x4_t hi = split(x), mid = split(x), lo = split(x);
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) {
        const u32x4_t kt = __builtin_bit_cast(u32x4_t, KB::cols(ka, st, i));
        S[i] = mfma(kt, hi, S[i]);
        S[i] = mfma(kt, mid, S[i]);
        S[i] = mfma(kt, lo, S[i]);
      }
    }
    if constexpr (!STATE) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const int row = t + 32 * tt + lrow;
        if (row < t_hi) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            u32x2_t x = {pack_bf16x2(O[tt][4 * g], O[tt][4 * g + 1]), pack_bf16x2(O[tt][4 * g + 2], O[tt][4 * g + 3])};
            if (row >= len) x = u32x2_t{};
            *reinterpret_cast<u32x2_t *>(o_ + row * o_stride + 8 * g + 4 * half) = x;
          }
        }
      }
    }
    lds_barrier();  // everyone is done with the chunk
    if (t + kC < t_end) load_chunk(t + kC);
  }
  if constexpr (!STATE) {
    // rows behind the sequence, from the first whole chunk on
    const int z0 = t_lo < t_end ? t_lo + (t_end - t_lo + kC - 1) / kC * kC : t_lo;
    for (long long i = z0 * 4LL + lane; i < t_hi * 4LL; i += 64)
      *reinterpret_cast<u32x4_t *>(o_ + static_cast<size_t>(i >> 2) * o_stride + 8 * static_cast<int>(i & 3)) = u32x4_t{};
    if (!a.s_out || seg != a.segs - 1) return;
  } else if (tid == 0 && slice == 0) {
    a.sums[head * (a.segs - 1) + seg] = total;
  }
  float *const to = (STATE ? a.seg + (head * a.segs + seg + 1) * dkv : a.s_out + head * dkv) + col;
#pragma unroll
  for (int i = 0; i < DK / 32; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) to[static_cast<size_t>(32 * i + 8 * (e >> 2) + 4 * half + (e & 3)) * a.dv] = S[i][e];
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
  const int n = a.segs - 1;
  float *const own = a.seg + head * a.segs * dkv + at;
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

// One token: workgroup = (sequence, head, `cols` of the values), the state read and written once. A row of the slice
// is cols / 4 lanes' 16 bytes; rows are dealt to the lane groups, whose shares of o meet in LDS.
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
  const float keep = __builtin_amdgcn_exp2f(log2_decay(g));
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

// Segments of a prompt: as many as give the chip two workgroups a CU, of four chunks at least.
LinearPlan linear_plan(int B, int T, int H, int dv) {
  const long long groups = static_cast<long long>(B) * H * (dv == 64 ? 1 : dv / 128);
  const int chunks = (T + kC - 1) / kC;
  long long segs = std::max<long long>(512 / groups, 1);
  segs = std::min<long long>(segs, std::max(chunks / 4, 1));
  LinearPlan p;
  p.seg_len = static_cast<int>((chunks + segs - 1) / segs) * kC;
  p.segs = (T + p.seg_len - 1) / p.seg_len;
  return p;
}

namespace {

template <int DK, int DVS> hipError_t launch(LinearArgs a, hipStream_t s) {
  const long long rows = static_cast<long long>(a.B) * a.H * (a.dv / DVS);
  if (a.segs > 1) {
    a.run = a.segs - 1;
    const long long g = rows * a.run;
    linear_fwd<DK, DVS, true><<<dim3(grid_x(g), grid_rows(g)), DVS * 2, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long c = (static_cast<long long>(a.B) * a.H * DK * (a.dv / 4) + 255) / 256;
    linear_carry<<<dim3(grid_x(c), grid_rows(c)), 256, 0, s>>>(a);
    const hipError_t f = hipGetLastError();
    if (f != hipSuccess) return f;
  }
  a.run = a.segs;
  const long long g = rows * a.run;
  linear_fwd<DK, DVS, false><<<dim3(grid_x(g), grid_rows(g)), DVS * 2, 0, s>>>(a);
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
  // few rows: narrow slices, so that more workgroups share them
  const long long rows = static_cast<long long>(a.N) * a.H;
  if (a.dv == 64 || rows * (a.dv / 64) <= 1024) return rows * (a.dv / 64) > 256 ? launch<64>(a, s) : launch<32>(a, s);
  return a.dv == 128 ? launch<128>(a, s) : launch<256>(a, s);
}

}  // namespace rglru
