// rglru_mqa_bwd.hip -- gradients of local attention (rglru_local_attention), bf16 on gfx950.
//
// With s = q k^T, p = exp(scale s - lse) on the visible pairs (0 elsewhere), and given do = dL/do:
//   delta_t = <do_t, o_t>,  dp = do v^T,  ds = p (dp - delta),
//   dq = scale ds k,  dk = scale sum_heads ds^T q,  dv = sum_heads p^T do.
//
// Two kernels, each recomputing p, with no floating-point atomics (bitwise reproducible):
//   attn_dq   owns 128 rows of one query head (a wave 32) and walks the key blocks they see; q and do
//             are in registers, K and V blocks in LDS: S^T = K Q^T, dP^T = V dO^T,
//             dQ^T += K^T dS^T. It also forms delta, which the second kernel reads.
//   attn_dkv  owns 128 keys (a wave 32) and walks (head of the group, block of 64 rows) items that
//             see them; k and v are in registers, Q and dO blocks in LDS: S = Q K^T, dP = dO V^T,
//             dV^T += dO^T P, dK^T += Q^T dS.
// In both, the accumulator layout of S and dP (one column per lane, 16 rows) is already the B
// operand's of the products that follow, if these take their k index in the accumulator's order:
// P and dS never leave the registers. The other operand of those products is a transpose of a block
// in LDS, read by ds_read_b64_tr_b16. Blocks arrive by direct buffer-to-LDS loads, two buffers, one
// barrier per block. The 16-byte chunk c of row r lies at c ^ f(r), with f chosen so that both the
// row reads (16 consecutive rows at one chunk) and the transposing reads (4 consecutive rows at 4
// consecutive chunks) of a pass fall on different banks.
//
// Key blocks that many rows see (all heads of a group; sinks: all rows after them) are split over
// several workgroups, whose fp32 partial dK and dV attn_dkv_sum adds in order.
#include "rglru_launch.h"
#include "rglru_mfma.h"

#include <algorithm>
#include <type_traits>

namespace rglru {

namespace {

constexpr int kRawWord3 = 0x00020000;  // buffer descriptor word 3: raw 32-bit data, no swizzle
constexpr float kLn2Inv = 1.4426950408889634f;

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWg = 4;         // waves per workgroup
constexpr int kOwn = 32 * kWg; // rows (attn_dq) or keys (attn_dkv) per workgroup
constexpr int kBlk = 64;       // rows per LDS block
constexpr int kFewKeys = 256;  // rows with fewer keys: delta from the sums, not from o

// A block of kBlk rows of DH bf16 in LDS, and the ways it is filled and read.
template <int DH> struct Blk {
  static constexpr int kElems = kBlk * DH;
  static constexpr int kCPR = DH / 8;                 // 16-byte chunks per row
  static constexpr int kRPI = 64 / kCPR;              // rows per wave-wide 16-byte load
  static constexpr int kLPW = kBlk / kRPI / kWg;      // loads per wave
  static constexpr int kKS = DH / 16;                 // k-steps over d
  static constexpr int kDT = DH / 32;                 // 32-wide d tiles
  // chunk swizzle: rows of 128 bytes (DH 64) share a 256-byte bank line in pairs
  __device__ __forceinline__ static int swz(int r) {
    return DH == 64 ? 4 * ((r >> 1) & 1) + ((r >> 2) & 3) : 4 * (r & 3) + ((r >> 2) & 3);
  }
  // the buffer of a block's rows: those of the sequence from `base` on, at most kBlk (rows past its
  // end then read zero, whatever lies there)
  __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rsrc(const bf16_t *base,
                                                                unsigned row_bytes, int rows) {
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<bf16_t *>(wave_uniform(base)), static_cast<short>(0),
        static_cast<int>(row_bytes * static_cast<unsigned>(min(rows, kBlk) - 1)) + DH * 2, kRawWord3);
  }
  // this wave's ii-th load of the block's rows to dst
  __device__ __forceinline__ static void load(__amdgpu_buffer_rsrc_t src, unsigned row_bytes,
                                              int ii, int w, int lane, const bf16_t *dst) {
    const int i = w + kWg * ii;
    const int row = i * kRPI + lane / kCPR;
    const unsigned off = static_cast<unsigned>(row) * row_bytes +
                         static_cast<unsigned>(((lane % kCPR) ^ swz(row)) * 16);
    dma_16b(src, off, lds_addr(dst + i * 512));
  }
  // A operand, rows 32 hf.., k = d of step s: 8 values of row lane % 32
  __device__ __forceinline__ static bf16x8_t rows(const bf16_t *b, int hf, int s, int lane) {
    const int r = lane & 31;
    return load_bf16x8(b + (32 * hf + r) * DH + (((2 * s + (lane >> 5)) ^ swz(r)) * 8));
  }
  // A operand, rows d = 32 j + lane % 32, k = block rows 32 hf + 16 st + (4 h.., 8 + 4 h..), h =
  // lane / 32: the accumulator's row order
  __device__ __forceinline__ static bf16x8_t cols(const bf16_t *b, int hf, int st, int j, int lane) {
    const int half = lane >> 5, r4 = (lane & 15) >> 2;
    const int cl = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int rj = DH == 64 ? r4 >> 1 : r4;
    const bf16_t *p = b + (32 * hf + 16 * st + 4 * half + r4) * DH + 32 * (j ^ rj) + 4 * (lane & 1);
    const i16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(p + 8 * (cl ^ half)));
    const i16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_i16x4_t *)(p + 8 * DH + 8 * (cl ^ half ^ 2)));
    const uint2 ux = __builtin_bit_cast(uint2, x), uy = __builtin_bit_cast(uint2, y);
    const u32x4_t u = {ux.x, ux.y, uy.x, uy.y};
    return __builtin_bit_cast(bf16x8_t, u);
  }
};

// Key row kr sees query row t (t, kr < len checked apart).
__device__ __forceinline__ bool sees(int t, int u, int W, int sinks) {
  return u <= t && (u > t - W || u < sinks);
}

__device__ __forceinline__ int clamp_len(const int *lens, int b, int T) {
  return lens ? min(max(lens[b], 0), T) : T;
}

}  // namespace

template <int DH>
__global__ __launch_bounds__(64 * kWg, DH == 256 ? 1 : 2) void attn_dq(AttnBwdArgs a) {
  typedef Blk<DH> K;
  __shared__ __attribute__((aligned(16))) bf16_t smem[4 * K::kElems];  // K[2], V[2]
  bf16_t *const Kb = smem, *const Vb = smem + 2 * K::kElems;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lrow = lane & 31, half = lane >> 5;
  const int T = a.T, Hq = a.Hq, W = a.window, sinks = a.sinks;
  // heavy first: query blocks from the last one down, all (sequence, head) pairs of one together
  const int nbh = a.B * Hq;
  const int nqb = (T + kOwn - 1) / kOwn;
  const int qi = blockIdx.x / nbh, bh = blockIdx.x - qi * nbh;
  const int q0 = (nqb - 1 - qi) * kOwn;
  const int h = bh % Hq, b = bh / Hq;
  const int len = clamp_len(a.lens, b, T);
  const int qw = q0 + 32 * w, qr = qw + lrow;
  const size_t tok = static_cast<size_t>(b) * T;
  const int qc = min(qr, T - 1);
  float *const delta = a.delta + (static_cast<size_t>(b) * Hq + h) * T;
  bf16_t *const dq = static_cast<bf16_t *>(a.dq) + (tok + qc) * a.dq_stride + static_cast<size_t>(h) * DH;
  if (q0 >= len) {
    if (qr < T) {
#pragma unroll
      for (int s = 0; s < K::kKS; ++s) *reinterpret_cast<u32x4_t *>(dq + 16 * s + 8 * half) = u32x4_t{};
      if (half == 0) delta[qr] = 0.0f;
    }
    return;
  }
  // this lane's row: q and do as B operands, delta = <do, o>
  bf16x8_t qf[K::kKS], gf[K::kKS];
  float dl = 0.0f;
  {
    const bf16_t *qp = static_cast<const bf16_t *>(a.q) + (tok + qc) * a.q_stride +
                       static_cast<size_t>(h) * DH + 8 * half;
    const size_t oo = ((tok + qc) * Hq + h) * DH + 8 * half;
    const bf16_t *gp = static_cast<const bf16_t *>(a.do_) + oo;
    const bf16_t *op = static_cast<const bf16_t *>(a.o) + oo;
#pragma unroll
    for (int s = 0; s < K::kKS; ++s) {
      qf[s] = load_bf16x8(qp + 16 * s);
      gf[s] = load_bf16x8(gp + 16 * s);
      const u32x4_t g = __builtin_bit_cast(u32x4_t, gf[s]);
      const u32x4_t o = *reinterpret_cast<const u32x4_t *>(op + 16 * s);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dl = fmaf(bf16lo(g[e]), bf16lo(o[e]), fmaf(bf16hi(g[e]), bf16hi(o[e]), dl));
    }
    dl += __shfl_xor(dl, 32, 64);
  }
  const bool in = qr < len;
  const float l2 = in ? a.lse[(static_cast<size_t>(b) * Hq + h) * T + qc] * kLn2Inv : __builtin_inff();
  // complete these loads here: the compiler does not see the LDS loads that share their counter
#pragma unroll
  for (int s = 0; s < K::kKS; ++s) asm volatile("" ::"v"(qf[s]), "v"(gf[s]));

  const int kvh = h / a.group;
  const bf16_t *kb_ = static_cast<const bf16_t *>(a.k) + tok * a.k_stride + static_cast<size_t>(kvh) * DH;
  const bf16_t *vb_ = static_cast<const bf16_t *>(a.v) + tok * a.v_stride + static_cast<size_t>(kvh) * DH;
  const unsigned krb = static_cast<unsigned>(a.k_stride) * 2, vrb = static_cast<unsigned>(a.v_stride) * 2;
  // the walk: blocks with sinks before the window's first block, then the window's
  const int last = min(len, q0 + kOwn) - 1;
  const int win = max(0, q0 - W + 1) / kBlk, end = last / kBlk + 1;
  const int ns = min((sinks + kBlk - 1) / kBlk, win);
  const int n = ns + end - win;
  auto first_row = [&](int i) { return (i < ns ? i : i - ns + win) * kBlk; };
  auto load_block = [&](int i) {
    const int u0 = first_row(i), buf = (i & 1) * K::kElems;
    const __amdgpu_buffer_rsrc_t ks = K::rsrc(kb_ + static_cast<size_t>(u0) * a.k_stride, krb, len - u0);
    const __amdgpu_buffer_rsrc_t vs = K::rsrc(vb_ + static_cast<size_t>(u0) * a.v_stride, vrb, len - u0);
#pragma unroll
    for (int ii = 0; ii < K::kLPW; ++ii) {
      K::load(ks, krb, ii, w, lane, Kb + buf);
      K::load(vs, vrb, ii, w, lane, Vb + buf);
    }
  };
  f32x16_t acc[K::kDT];
#pragma unroll
  for (int j = 0; j < K::kDT; ++j) acc[j] = f32x16_t{};
  const bool one = W == 1 && sinks == 0;
  // one walk over the blocks; kDelta: only the sums of p dp and of p
  float sp = 0.0f, spd = 0.0f;
  auto walk = [&](auto delta_only) {
    constexpr bool kDelta = decltype(delta_only)::value;
    load_block(0);
    for (int i = 0; i < n; ++i) {
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's rows of block i landed
      lds_barrier();                        // everyone's landed; everyone is done with block i - 1
      if (i + 1 < n) load_block(i + 1);
      const bf16_t *Kc = Kb + (i & 1) * K::kElems, *Vc = Vb + (i & 1) * K::kElems;
      const int u0 = first_row(i);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int U = u0 + 32 * hf;
        // some pair of (my rows, these keys) visible?
        if (U > qw + 31 || (U + 31 <= qw - W && U >= sinks) || qw >= len) continue;
        f32x16_t s = f32x16_t{}, dp = f32x16_t{};
#pragma unroll
        for (int d = 0; d < K::kKS; ++d)
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(K::rows(Kc, hf, d, lane), qf[d], s, 0, 0, 0);
#pragma unroll
        for (int d = 0; d < K::kKS; ++d)
          dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(K::rows(Vc, hf, d, lane), gf[d], dp, 0, 0, 0);
        const bool full = U + 31 <= qw && (U > qw + 31 - W || U + 31 < sinks);  // U + 31 < len follows
        if (!full) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int u = U + 8 * (e >> 2) + 4 * half + (e & 3);
            s[e] = sees(qr, u, W, sinks) && u < len ? s[e] : -__builtin_inff();
            dp[e] = one || qr == 0 ? dl : dp[e];  // a row with one key has no gradient
          }
        }
        if constexpr (kDelta) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[e], a.c, -l2));
            sp += p;
            spd = fmaf(p, dp[e], spd);
          }
        } else {
          u32x4_t ds[2];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float p0 = __builtin_amdgcn_exp2f(fmaf(s[e], a.c, -l2));
            const float p1 = __builtin_amdgcn_exp2f(fmaf(s[e + 1], a.c, -l2));
            ds[e >> 3][(e >> 1) & 3] = pack_bf16x2(p0 * (dp[e] - dl), p1 * (dp[e + 1] - dl));
          }
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int j = 0; j < K::kDT; ++j)
              acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                  K::cols(Kc, hf, st, j, lane), __builtin_bit_cast(bf16x8_t, ds[st]), acc[j], 0, 0, 0);
        }
      }
    }
  };
  // delta from the rounded o is off by a 2^-9th of its terms, which averages out over many keys but
  // not over few, where dp - delta is a small difference: row blocks with fewer than kFewKeys keys
  // in some row take it as sum p dp / sum p instead, in a walk of its own.
  if (min(q0 + 1, W) < kFewKeys) {
    walk(std::true_type{});
    sp += __shfl_xor(sp, 32, 64);
    spd += __shfl_xor(spd, 32, 64);
    dl = spd / sp;
    lds_barrier();  // the buffers are filled again
  }
  if (half == 0 && qr < T) delta[qr] = in ? dl : 0.0f;
  walk(std::false_type{});
  if (qr >= T) return;
  const float f = in ? a.scale : 0.0f;
#pragma unroll
  for (int j = 0; j < K::kDT; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint2 v = make_uint2(pack_bf16x2(acc[j][4 * g] * f, acc[j][4 * g + 1] * f),
                           pack_bf16x2(acc[j][4 * g + 2] * f, acc[j][4 * g + 3] * f));
      if (!in) v = make_uint2(0u, 0u);
      *reinterpret_cast<uint2 *>(dq + 32 * j + 8 * g + 4 * half) = v;
    }
}

// Key block kb of a sequence: [64-row query blocks that see it], for the static length T; the
// splits of blocks with sinks and of the others are a.s_sink and a.s_win.
template <int DH>
__global__ __launch_bounds__(64 * kWg, DH == 256 ? 1 : 2) void attn_dkv(AttnBwdArgs a) {
  typedef Blk<DH> K;
  __shared__ __attribute__((aligned(16))) bf16_t smem[4 * K::kElems];  // Q[2], dO[2]
  __shared__ __attribute__((aligned(16))) float rowv[2][2][kBlk];      // [buffer][lse, delta][row]
  bf16_t *const Qb = smem, *const Gb = smem + 2 * K::kElems;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lrow = lane & 31, half = lane >> 5;
  const int T = a.T, Hq = a.Hq, W = a.window, sinks = a.sinks;
  const int bk = blockIdx.x / a.slots, slot = blockIdx.x - bk * a.slots;
  const int kvh = bk % a.Hkv, b = bk / a.Hkv;
  const int head_slots = a.nsb * a.s_sink;
  int kb, sp, S;
  if (slot < head_slots) {
    S = a.s_sink;
    kb = slot / S;
    sp = slot - kb * S;
  } else {
    S = a.s_win;
    kb = (slot - head_slots) / S;
    sp = slot - head_slots - kb * S;
    kb += a.nsb;
  }
  const int K0 = kb * kOwn;
  const int len = clamp_len(a.lens, b, T);
  const int kw = K0 + 32 * w, kr = kw + lrow;
  const size_t tok = static_cast<size_t>(b) * T;
  // this lane's key: k and v as B operands (rows past the sequence: zero)
  bf16x8_t kf[K::kKS], vf[K::kKS];
  {
    const size_t row = tok + min(kr, T - 1);
    const bf16_t *kp = static_cast<const bf16_t *>(a.k) + row * a.k_stride + static_cast<size_t>(kvh) * DH + 8 * half;
    const bf16_t *vp = static_cast<const bf16_t *>(a.v) + row * a.v_stride + static_cast<size_t>(kvh) * DH + 8 * half;
    const bool in = kr < len;
#pragma unroll
    for (int s = 0; s < K::kKS; ++s) {
      u32x4_t x = *reinterpret_cast<const u32x4_t *>(kp + 16 * s);
      u32x4_t y = *reinterpret_cast<const u32x4_t *>(vp + 16 * s);
      if (!in) x = y = u32x4_t{};
      kf[s] = __builtin_bit_cast(bf16x8_t, x);
      vf[s] = __builtin_bit_cast(bf16x8_t, y);
    }
#pragma unroll
    for (int s = 0; s < K::kKS; ++s) asm volatile("" ::"v"(kf[s]), "v"(vf[s]));
  }
  f32x16_t dk[K::kDT], dv[K::kDT];
#pragma unroll
  for (int j = 0; j < K::kDT; ++j) dk[j] = dv[j] = f32x16_t{};
  // items: (head of the group, 64-row block); this workgroup's share
  const int qfirst = K0 / kBlk;
  const int qlast_row = K0 < sinks ? len - 1
                                   : static_cast<int>(min(static_cast<long long>(len) - 1,
                                                          static_cast<long long>(K0) + kOwn - 2 + W));
  const int nq = K0 < len ? qlast_row / kBlk - qfirst + 1 : 0;
  const int items = nq * a.group;
  const int share = (items + S - 1) / S;
  const int i0 = min(items, sp * share), i1 = min(items, i0 + share);
  const unsigned qrb = static_cast<unsigned>(a.q_stride) * 2, grb = static_cast<unsigned>(Hq) * DH * 2;
  const bf16_t *qb_ = static_cast<const bf16_t *>(a.q) + tok * a.q_stride;
  const bf16_t *gb_ = static_cast<const bf16_t *>(a.do_) + tok * Hq * DH;
  const bool one = W == 1 && sinks == 0;
  float pre = 0.0f;  // threads 0..127: the next block's lse or delta
  auto load_item = [&](int i) {
    const int hh = i / nq, q0 = (qfirst + i - hh * nq) * kBlk, buf = (i & 1) * K::kElems;
    const int h = kvh * a.group + hh;
    const __amdgpu_buffer_rsrc_t qs =
        K::rsrc(qb_ + static_cast<size_t>(q0) * a.q_stride + static_cast<size_t>(h) * DH, qrb, len - q0);
    const __amdgpu_buffer_rsrc_t gs =
        K::rsrc(gb_ + (static_cast<size_t>(q0) * Hq + h) * DH, grb, len - q0);
#pragma unroll
    for (int ii = 0; ii < K::kLPW; ++ii) {
      K::load(qs, qrb, ii, w, lane, Qb + buf);
      K::load(gs, grb, ii, w, lane, Gb + buf);
    }
    if (tid < 2 * kBlk) {
      const int t = q0 + (tid & (kBlk - 1));
      const size_t at = (static_cast<size_t>(b) * Hq + h) * T + min(t, T - 1);
      if (tid < kBlk)
        pre = t < len ? a.lse[at] * kLn2Inv : __builtin_inff();
      else
        pre = t < len ? a.delta[at] : 0.0f;
    }
  };
  auto put_rows = [&](int i) {
    if (tid < 2 * kBlk) rowv[i & 1][tid / kBlk][tid & (kBlk - 1)] = pre;
  };
  if (i0 < i1) {
    load_item(i0);
    put_rows(i0);
  }
  for (int i = i0; i < i1; ++i) {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's rows of item i landed
    lds_barrier();
    if (i + 1 < i1) load_item(i + 1);
    const bf16_t *Qc = Qb + (i & 1) * K::kElems, *Gc = Gb + (i & 1) * K::kElems;
    const int hh = i / nq, q0 = (qfirst + i - hh * nq) * kBlk;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int Q = q0 + 32 * hf;
      if (kw > Q + 31 || (kw + 31 <= Q - W && kw >= sinks) || Q >= len || kw >= len) continue;
      f32x16_t s = f32x16_t{}, dp = f32x16_t{};
#pragma unroll
      for (int d = 0; d < K::kKS; ++d)
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(K::rows(Qc, hf, d, lane), kf[d], s, 0, 0, 0);
#pragma unroll
      for (int d = 0; d < K::kKS; ++d)
        dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(K::rows(Gc, hf, d, lane), vf[d], dp, 0, 0, 0);
      const bool full = kw + 31 <= Q && (kw > Q + 31 - W || kw + 31 < sinks);
      if (!full) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int t = Q + 8 * (e >> 2) + 4 * half + (e & 3);
          s[e] = sees(t, kr, W, sinks) ? s[e] : -__builtin_inff();
          // a row with one key has no gradient
          if (one || t == 0) dp[e] = rowv[i & 1][1][32 * hf + 8 * (e >> 2) + 4 * half + (e & 3)];
        }
      }
      u32x4_t pp[2], ds[2];
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const f32x4_t l2 = *reinterpret_cast<const f32x4_t *>(&rowv[i & 1][0][32 * hf + 8 * e4 + 4 * half]);
        const f32x4_t dl = *reinterpret_cast<const f32x4_t *>(&rowv[i & 1][1][32 * hf + 8 * e4 + 4 * half]);
        float p[4], d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = __builtin_amdgcn_exp2f(fmaf(s[4 * e4 + e], a.c, -l2[e]));
          d[e] = p[e] * (dp[4 * e4 + e] - dl[e]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          pp[e4 >> 1][2 * (e4 & 1) + e] = pack_bf16x2(p[2 * e], p[2 * e + 1]);
          ds[e4 >> 1][2 * (e4 & 1) + e] = pack_bf16x2(d[2 * e], d[2 * e + 1]);
        }
      }
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int j = 0; j < K::kDT; ++j)
          dv[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              K::cols(Gc, hf, st, j, lane), __builtin_bit_cast(bf16x8_t, pp[st]), dv[j], 0, 0, 0);
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int j = 0; j < K::kDT; ++j)
          dk[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              K::cols(Qc, hf, st, j, lane), __builtin_bit_cast(bf16x8_t, ds[st]), dk[j], 0, 0, 0);
    }
    if (i + 1 < i1) put_rows(i + 1);
  }
  // lane = key kr; accumulator e of tile j is d = 32 j + 8 (e / 4) + 4 half + e % 4
  if (S > 1) {
    float *pk = a.part + (static_cast<size_t>(blockIdx.x) * 2 * kOwn + (32 * w + lrow)) * DH + 4 * half;
    float *pv = pk + static_cast<size_t>(kOwn) * DH;
#pragma unroll
    for (int j = 0; j < K::kDT; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t x = {dk[j][4 * g], dk[j][4 * g + 1], dk[j][4 * g + 2], dk[j][4 * g + 3]};
        const f32x4_t y = {dv[j][4 * g], dv[j][4 * g + 1], dv[j][4 * g + 2], dv[j][4 * g + 3]};
        *reinterpret_cast<f32x4_t *>(pk + 32 * j + 8 * g) = x;
        *reinterpret_cast<f32x4_t *>(pv + 32 * j + 8 * g) = y;
      }
    return;
  }
  if (kr >= T) return;
  bf16_t *ok = static_cast<bf16_t *>(a.dk) + (tok + kr) * a.dk_stride + static_cast<size_t>(kvh) * DH + 4 * half;
  bf16_t *ov = static_cast<bf16_t *>(a.dv) + (tok + kr) * a.dv_stride + static_cast<size_t>(kvh) * DH + 4 * half;
#pragma unroll
  for (int j = 0; j < K::kDT; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float f = a.scale;
      *reinterpret_cast<uint2 *>(ok + 32 * j + 8 * g) =
          make_uint2(pack_bf16x2(dk[j][4 * g] * f, dk[j][4 * g + 1] * f),
                     pack_bf16x2(dk[j][4 * g + 2] * f, dk[j][4 * g + 3] * f));
      *reinterpret_cast<uint2 *>(ov + 32 * j + 8 * g) =
          make_uint2(pack_bf16x2(dv[j][4 * g], dv[j][4 * g + 1]),
                     pack_bf16x2(dv[j][4 * g + 2], dv[j][4 * g + 3]));
    }
}

// dk, dv of the split key blocks: the partial sums in order, 8 values per lane.
__global__ __launch_bounds__(256) void attn_dkv_sum(AttnBwdArgs a, int dh) {
  const int cpr = dh / 8;
  const size_t per = static_cast<size_t>(a.T) * cpr;  // lanes per (sequence, head, which)
  const size_t total = per * a.B * a.Hkv * 2;
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const size_t bkw = i / per, r = i - bkw * per;
  const int which = static_cast<int>(bkw & 1);
  const size_t bk = bkw >> 1;
  const int t = static_cast<int>(r / cpr), c = static_cast<int>(r - static_cast<size_t>(t) * cpr);
  const int kb = t / kOwn;
  const bool sink = kb < a.nsb;
  const int S = sink ? a.s_sink : a.s_win;
  if (S == 1) return;
  const int slot = sink ? kb * S : a.nsb * a.s_sink + (kb - a.nsb) * S;
  const float *p = a.part + (((bk * a.slots + slot) * 2 + which) * kOwn + (t - kb * kOwn)) * dh + c * 8;
  float acc[8] = {};
  for (int s = 0; s < S; ++s, p += static_cast<size_t>(2) * kOwn * dh) {
    const f32x4_t x = *reinterpret_cast<const f32x4_t *>(p), y = *reinterpret_cast<const f32x4_t *>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[e] += x[e];
      acc[4 + e] += y[e];
    }
  }
  const float f = which ? 1.0f : a.scale;
  u32x4_t v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = pack_bf16x2(acc[2 * e] * f, acc[2 * e + 1] * f);
  const int b = static_cast<int>(bk / a.Hkv), kvh = static_cast<int>(bk % a.Hkv);
  bf16_t *out = static_cast<bf16_t *>(which ? a.dv : a.dk) +
                (static_cast<size_t>(b) * a.T + t) * (which ? a.dv_stride : a.dk_stride) +
                static_cast<size_t>(kvh) * dh + c * 8;
  *reinterpret_cast<u32x4_t *>(out) = v;
}

// Splits of the key blocks: enough workgroups for the chip, shares of about equal length.
AttnBwdPlan attn_bwd_plan(int B, int T, int Hq, int Hkv, int window, int sinks) {
  AttnBwdPlan p;
  const int nkb = (T + kOwn - 1) / kOwn;
  p.nsb = std::min((std::min(sinks, T) + kOwn - 1) / kOwn, nkb);
  const int group = Hq / Hkv;
  const long long q_all = (T + kBlk - 1) / kBlk;
  const long long q_win = std::min<long long>(q_all, (kOwn + static_cast<long long>(window) + kBlk - 2) / kBlk + 1);
  const long long items = (p.nsb * q_all + (nkb - p.nsb) * q_win) * group * B * Hkv;
  constexpr long long kTarget = 512;  // workgroups
  const long long share = std::max<long long>(4, (items + kTarget - 1) / kTarget);
  p.s_sink = static_cast<int>(std::max<long long>(1, (q_all * group + share / 2) / share));
  p.s_win = static_cast<int>(std::max<long long>(1, (q_win * group + share / 2) / share));
  p.slots = p.nsb * p.s_sink + (nkb - p.nsb) * p.s_win;
  return p;
}
size_t attn_bwd_delta_floats(int B, int T, int Hq) { return static_cast<size_t>(B) * T * Hq; }
size_t attn_bwd_part_floats(const AttnBwdPlan &p, int B, int Hkv, int dh) {
  if (p.s_sink == 1 && p.s_win == 1) return 0;
  return static_cast<size_t>(B) * Hkv * p.slots * 2 * kOwn * dh;
}

namespace {

template <int DH> hipError_t launch(const AttnBwdArgs &a, hipStream_t s) {
  const unsigned nq = static_cast<unsigned>((a.T + kOwn - 1) / kOwn);
  attn_dq<DH><<<nq * a.B * a.Hq, 64 * kWg, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  attn_dkv<DH><<<static_cast<unsigned>(a.slots) * a.B * a.Hkv, 64 * kWg, 0, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || (a.s_sink == 1 && a.s_win == 1)) return e;
  const size_t n = static_cast<size_t>(a.T) * (DH / 8) * a.B * a.Hkv * 2;
  attn_dkv_sum<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(a, DH);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_local_attention_backward(const AttnBwdArgs &a, int dh, hipStream_t s) {
  switch (dh) {
    case 64: return launch<64>(a, s);
    case 128: return launch<128>(a, s);
    case 256: return launch<256>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace rglru
