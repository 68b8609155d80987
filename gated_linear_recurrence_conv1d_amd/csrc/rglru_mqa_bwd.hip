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
// in LDS, read by ds_read_b64_tr_b16. Blocks of 32 rows arrive by direct buffer-to-LDS loads, two ahead,
// in a ring of four: the products with a transposed operand lag by one block, so that they run on the
// matrix cores beside the next block's exponentials (one wave per SIMD at dh 256: nothing else would
// fill them). One barrier per block. The 16-byte chunk c of row r lies at c ^ f(r), with f chosen so that both the
// row reads (16 consecutive rows at one chunk) and the transposing reads (4 consecutive rows at 4
// consecutive chunks) of a pass fall on different banks.
//
// Key blocks that many rows see (all heads of a group; sinks: all rows after them) are split over
// several workgroups, whose fp32 partial dK and dV attn_dkv_sum adds in order.
#include "rglru_attn.h"
#include "rglru_launch.h"

#include <algorithm>
#include <type_traits>

namespace rglru {

using namespace attn;

namespace {

constexpr int kRing = 4;       // attn_dq's blocks in LDS: the last one, this one and two on their way
constexpr int kFewKeys = 256;  // rows with fewer keys: delta from the sums, not from o

}  // namespace

template <int DH>
__global__ __launch_bounds__(64 * kWg, DH == 256 ? 1 : 2) void attn_dq(AttnBwdArgs a) {
  typedef Blk<DH> K;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[kRing * K::kSlot];
  const unsigned lds = lds_addr(smem);
  auto slot_of = [&](int i) { return lds + (i & (kRing - 1)) * K::kSlot; };
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lrow = lane & 31, half = lane >> 5;
  const int T = a.T, Hq = a.Hq, W = a.window, sinks = a.sinks;
  // heavy first: query blocks from the last one down, all (sequence, head) pairs of one together
  const int nbh = a.B * Hq;
  const int nqb = (T + kOwn - 1) / kOwn;
  const int qi = uni(blockIdx.x / nbh), bh = blockIdx.x - qi * nbh;
  const int q0 = (nqb - 1 - qi) * kOwn;
  const int b = uni(bh / Hq), h = bh - b * Hq;
  const int len = clamp_len(a.lens, b, T);
  const int qw = q0 + 32 * w, qr = qw + lrow;
  const size_t tok = static_cast<size_t>(b) * T;
  const int qc = min(qr, T - 1);
  float2 *const stat = a.stat + (static_cast<size_t>(b) * Hq + h) * T;
  bf16_t *const dq = static_cast<bf16_t *>(a.dq) + (tok + qc) * a.dq_stride + static_cast<size_t>(h) * DH;
  if (q0 >= len) {
    if (qr < T) {
#pragma unroll
      for (int s = 0; s < K::kKS; ++s) *reinterpret_cast<u32x4_t *>(dq + 16 * s + 8 * half) = u32x4_t{};
      if (half == 0) stat[qr] = make_float2(__builtin_inff(), 0.0f);
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

  const int kvh = uni(h / a.group);
  const bf16_t *kb_ = static_cast<const bf16_t *>(a.k) + tok * a.k_stride + static_cast<size_t>(kvh) * DH;
  const bf16_t *vb_ = static_cast<const bf16_t *>(a.v) + tok * a.v_stride + static_cast<size_t>(kvh) * DH;
  const unsigned krb = static_cast<unsigned>(a.k_stride) * 2, vrb = static_cast<unsigned>(a.v_stride) * 2;
  // the walk: blocks with sinks before the window's first block, then the window's
  const int last = min(len, q0 + kOwn) - 1;
  const int win = max(0, q0 - W + 1) / kBlk, end = last / kBlk + 1;
  const int ns = min((sinks + kBlk - 1) / kBlk, win);
  const int n = ns + end - win;
  auto first_row = [&](int i) { return (i < ns ? i : i - ns + win) * kBlk; };
  // the loads of block i (past the last one: zeros, without touching memory, so that every step
  // issues the same number)
  const typename K::Lane kl = K::load_lane(w, lane, krb), vl = K::load_lane(w, lane, vrb);
  struct Src {
    const bf16_t *k, *v;
    int rows;
  };
  auto src_of = [&](int i) {
    const int u0 = first_row(min(i, n - 1));
    return Src{kb_ + static_cast<size_t>(u0) * a.k_stride, vb_ + static_cast<size_t>(u0) * a.v_stride,
               i < n ? len - u0 : 0};
  };
  auto load_part = [&](const Src &src, int i, int ii) {
    const unsigned dst = slot_of(i);
    K::load(src.k, krb, src.rows, ii, w, kl, dst);
    K::load(src.v, vrb, src.rows, ii, w, vl, dst + K::kBytes);
  };
  auto load_block = [&](int i) {
    const Src src = src_of(i);
#pragma unroll
    for (int ii = 0; ii < K::kLPW; ++ii) load_part(src, i, ii);
  };
  const unsigned row_lane = K::row_lane(lane), col_lane = K::col_lane(lane);
  f32x16_t acc[K::kDT];
#pragma unroll
  for (int j = 0; j < K::kDT; ++j) acc[j] = f32x16_t{};
  const bool one = W == 1 && sinks == 0;
  // one walk over the blocks; kDelta: only the sums of p dp and of p
  float sp = 0.0f, spd = 0.0f;
  auto walk = [&](auto delta_only) {
    constexpr bool kDelta = decltype(delta_only)::value;
    load_block(0);
    load_block(1);
    u32x4_t ds[2] = {};  // the last block's dS
    for (int i = 0; i < n; ++i) {
      // this wave's rows of block i have landed (those of i + 1 may be on their way); then everyone's
      // have, and everyone is done with block i - 2
      __builtin_amdgcn_s_waitcnt(0x0F70 | (2 * K::kLPW));
      lds_barrier();
      const unsigned at = slot_of(i) + row_lane;
      const int U = first_row(i);
      f32x16_t s = f32x16_t{}, dp = f32x16_t{};
      const Src src = src_of(i + 2);
#pragma unroll
      for (int d = 0; d < K::kKS; ++d) {
        if (d % 4 == 0) load_part(src, i + 2, d / 4);
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(K::rows(at, d), qf[d], s, 0, 0, 0);
        dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(K::rows(at + K::kBytes, d), gf[d], dp, 0, 0, 0);
      }
      read_ahead<K::kKS, 2, 2, 3>();
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
        // the last block's dS^T into dQ^T beside this block's exponentials (block 0: zero into it)
        const unsigned pt = slot_of(i > 0 ? i - 1 : 0) + col_lane;
        u32x4_t dn[2];
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int j = 0; j < K::kDT; ++j)
            acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                K::cols(pt, st, j), __builtin_bit_cast(bf16x8_t, ds[st]), acc[j], 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float p0 = __builtin_amdgcn_exp2f(fmaf(s[e], a.c, -l2));
          const float p1 = __builtin_amdgcn_exp2f(fmaf(s[e + 1], a.c, -l2));
          dn[e >> 3][(e >> 1) & 3] = pack_bf16x2(p0 * (dp[e] - dl), p1 * (dp[e + 1] - dl));
        }
        ds[0] = dn[0];
        ds[1] = dn[1];
      }
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // the zeros have landed too
    if constexpr (!kDelta) {
      const unsigned pt = slot_of(n - 1) + col_lane;
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int j = 0; j < K::kDT; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              K::cols(pt, st, j), __builtin_bit_cast(bf16x8_t, ds[st]), acc[j], 0, 0, 0);
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
  if (half == 0 && qr < T) stat[qr] = make_float2(l2, in ? dl : 0.0f);
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

// Workgroup = 128 keys, 8 waves: wave (kt, side) has keys 32 kt.. . Side 0 holds k (B operands) and
// accumulates dV, side 1 holds v and accumulates dK, so that each fits in 256 registers and two waves,
// one of each side, share a SIMD:
//   step i, side 0: S(i) = Q K^T, P(i) = exp2(c S - lse), handed over through LDS; dV^T += dO^T P(i - 1)
//   step i, side 1: dP(i) = dO V^T; dS(i - 1) = P(i - 1) (dP(i - 1) - delta); dK^T += Q^T dS(i - 1)
// Both hold the same elements of S and dP in a lane, so the exchange is 16 values per lane, written and
// read in the lane's own order, and the one-step lag makes one barrier per step enough.
constexpr int kSlots = 3;  // blocks in LDS: the last one, this one, the next on its way
template <int DH> struct DkvLds {
  __attribute__((aligned(1024))) unsigned char blocks[kSlots * Blk<DH>::kSlot];
  f32x4_t px[2][kWg][4][64];       // P on its way to side 1
  float2 rowv[kSlots][kBlk];       // (lse in exp2 units, delta)
};

template <int DH, int SIDE>
__device__ __forceinline__ void dkv_side(const AttnBwdArgs &a, DkvLds<DH> &sh, int kt, int lane) {
  typedef Blk<DH> K;
  const unsigned lds = lds_addr(sh.blocks);
  const int lrow = lane & 31, half = lane >> 5;
  const int T = a.T, Hq = a.Hq, W = a.window, sinks = a.sinks;
  const int bk = uni(blockIdx.x / a.slots), wg_slot = blockIdx.x - bk * a.slots;
  const int b = uni(bk / a.Hkv), kvh = bk - b * a.Hkv;
  const int head_slots = a.nsb * a.s_sink;
  int kb, sp, S;
  if (wg_slot < head_slots) {
    S = a.s_sink;
    kb = uni(wg_slot / S);
    sp = wg_slot - kb * S;
  } else {
    S = a.s_win;
    kb = uni((wg_slot - head_slots) / S);
    sp = wg_slot - head_slots - kb * S;
    kb += a.nsb;
  }
  const int K0 = kb * kOwn;
  const int len = clamp_len(a.lens, b, T);
  const int kw = K0 + 32 * kt, kr = kw + lrow;
  const size_t tok = static_cast<size_t>(b) * T;
  // this lane's key: k or v as B operands (rows past the sequence: zero)
  bf16x8_t kf[K::kKS];
  {
    const bf16_t *kp = static_cast<const bf16_t *>(SIDE ? a.v : a.k) +
                       (tok + min(kr, T - 1)) * (SIDE ? a.v_stride : a.k_stride) +
                       static_cast<size_t>(kvh) * DH + 8 * half;
    const bool in = kr < len;
#pragma unroll
    for (int s = 0; s < K::kKS; ++s) {
      u32x4_t x = *reinterpret_cast<const u32x4_t *>(kp + 16 * s);
      if (!in) x = u32x4_t{};
      kf[s] = __builtin_bit_cast(bf16x8_t, x);
    }
#pragma unroll
    for (int s = 0; s < K::kKS; ++s) asm volatile("" ::"v"(kf[s]));
  }
  f32x16_t acc[K::kDT];  // dV^T or dK^T
#pragma unroll
  for (int j = 0; j < K::kDT; ++j) acc[j] = f32x16_t{};
  // items: (head of the group, 32-row block); this workgroup's share
  const int qfirst = K0 / kBlk;
  const int qlast_row = K0 < sinks ? len - 1
                                   : static_cast<int>(min(static_cast<long long>(len) - 1,
                                                          static_cast<long long>(K0) + kOwn - 2 + W));
  const int nq = K0 < len ? qlast_row / kBlk - qfirst + 1 : 0;
  const int items = nq * a.group;
  const int share = uni((items + S - 1) / S);
  const int i0 = min(items, sp * share), i1 = min(items, i0 + share);
  const bool one = W == 1 && sinks == 0;
  struct At {  // an item's head of the group and block
    int hh, qb;
  };
  auto next = [&](At &at) {
    if (++at.qb == nq) {
      at.qb = 0;
      ++at.hh;
    }
  };
  // side 0 brings the Q rows, side 1 the dO rows, and every wave the rows' stat
  const unsigned rb = SIDE ? static_cast<unsigned>(Hq) * DH * 2 : static_cast<unsigned>(a.q_stride) * 2;
  const bf16_t *const rows_ = static_cast<const bf16_t *>(SIDE ? a.do_ : a.q) + tok * (rb / 2);
  const typename K::Lane ll = K::load_lane(kt, lane, rb);
  auto load_item = [&](At at, int sl) {
    const int q0 = (qfirst + at.qb) * kBlk, h = kvh * a.group + at.hh;
    const __amdgpu_buffer_rsrc_t st = __builtin_amdgcn_make_buffer_rsrc(
        wave_uniform(a.stat + (static_cast<size_t>(b) * Hq + h) * T + q0), static_cast<short>(0),
        uni(min(len - q0, kBlk) * 8), kRawWord3);
#pragma unroll
    for (int ii = 0; ii < K::kLPW; ++ii)
      K::load(rows_ + static_cast<size_t>(q0) * (rb / 2) + static_cast<size_t>(h) * DH, rb, len - q0, ii, kt, ll,
              lds + sl * K::kSlot + (SIDE ? K::kBytes : 0u));
    dma_4b(st, lane * 4, lds_addr(sh.rowv[sl]));
  };
  const unsigned row_lane = K::row_lane(lane) + (SIDE ? K::kBytes : 0u);  // side 0 reads Q, 1 dO
  const unsigned col_lane = K::col_lane(lane) + (SIDE ? 0u : K::kBytes);  // side 0 reads dO, 1 Q
  u32x4_t pd[2] = {};         // P (side 0) or dS (side 1) of the last item
  // step i of the product into acc (row step i / kDT, d tile i % kDT; as many as S has k-steps)
  static_assert(2 * K::kDT == K::kKS, "one product step per k-step");
  auto product = [&](int sl, int i) {
    const int st = i / K::kDT, j = i % K::kDT;
    acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(K::cols(lds + sl * K::kSlot + col_lane, st, j),
                                                     __builtin_bit_cast(bf16x8_t, pd[st]), acc[j], 0, 0, 0);
  };
  f32x16_t dpl = f32x16_t{};  // side 1: dP of the last item
  // side 1: dS of the last item (first row Ql) from its P, dP and delta
  auto make_ds = [&](int buf, int sl, int Ql) {
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4) {
      const f32x4_t p = sh.px[buf][kt][e4][lane];
      const f32x4_t va = *reinterpret_cast<const f32x4_t *>(&sh.rowv[sl][8 * e4 + 4 * half]);
      const f32x4_t vb = *reinterpret_cast<const f32x4_t *>(&sh.rowv[sl][8 * e4 + 4 * half + 2]);
      float d[4] = {p[0] * (dpl[4 * e4] - va[1]), p[1] * (dpl[4 * e4 + 1] - va[3]),
                    p[2] * (dpl[4 * e4 + 2] - vb[1]), p[3] * (dpl[4 * e4 + 3] - vb[3])};
      if (one) d[0] = d[1] = d[2] = d[3] = 0.0f;  // a row with one key has no gradient
      if (Ql + 8 * e4 + 4 * half == 0) d[0] = 0.0f;
      pd[e4 >> 1][2 * (e4 & 1)] = pack_bf16x2(d[0], d[1]);
      pd[e4 >> 1][2 * (e4 & 1) + 1] = pack_bf16x2(d[2], d[3]);
    }
  };
  if (i0 < i1) {
    At cur = {uni(i0 / nq), 0};
    cur.qb = i0 - cur.hh * nq;
    At head = cur;
    int sl = 0, slp = 0;  // slots of this item and the last (the first one: its own, with P = 0)
    int Ql = 0;
    load_item(head, 0);
    for (int i = i0; i < i1; ++i) {
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's rows of item i landed
      lds_barrier();  // everyone's landed, everyone is done with item i - 2 and P(i - 1) is written
      const int sln = sl == kSlots - 1 ? 0 : sl + 1;
      next(head);
      if (i + 1 < i1) load_item(head, sln);
      const int Q = (qfirst + cur.qb) * kBlk;
      next(cur);
      if constexpr (SIDE == 1)
        if (i > i0) make_ds((i - 1) & 1, slp, Ql);
      f32x16_t s = f32x16_t{};
      const unsigned at = lds + sl * K::kSlot + row_lane;
#pragma unroll
      for (int d = 0; d < K::kKS; ++d) {
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(K::rows(at, d), kf[d], s, 0, 0, 0);
        product(slp, d);  // between the steps of S, which wait for each other
      }
      if constexpr (SIDE == 0) {
        const bool full = kw + 31 <= Q && (kw > Q + 31 - W || kw + 31 < sinks);
        if (!full) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int t = Q + 8 * (e >> 2) + 4 * half + (e & 3);
            s[e] = sees(t, kr, W, sinks) ? s[e] : -__builtin_inff();
          }
        }
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          const f32x4_t va = *reinterpret_cast<const f32x4_t *>(&sh.rowv[sl][8 * e4 + 4 * half]);
          const f32x4_t vb = *reinterpret_cast<const f32x4_t *>(&sh.rowv[sl][8 * e4 + 4 * half + 2]);
          const f32x4_t p = {__builtin_amdgcn_exp2f(fmaf(s[4 * e4], a.c, -va[0])),
                             __builtin_amdgcn_exp2f(fmaf(s[4 * e4 + 1], a.c, -va[2])),
                             __builtin_amdgcn_exp2f(fmaf(s[4 * e4 + 2], a.c, -vb[0])),
                             __builtin_amdgcn_exp2f(fmaf(s[4 * e4 + 3], a.c, -vb[2]))};
          sh.px[i & 1][kt][e4][lane] = p;
          pd[e4 >> 1][2 * (e4 & 1)] = pack_bf16x2(p[0], p[1]);
          pd[e4 >> 1][2 * (e4 & 1) + 1] = pack_bf16x2(p[2], p[3]);
        }
      } else {
        dpl = s;
      }
      Ql = Q;
      slp = sl;
      sl = sln;
    }
    lds_barrier();  // P of the last item
    if constexpr (SIDE == 1) make_ds((i1 - 1) & 1, slp, Ql);
#pragma unroll
    for (int d = 0; d < K::kKS; ++d) product(slp, d);
  }
  // lane = key kr; accumulator e of tile j is d = 32 j + 8 (e / 4) + 4 half + e % 4
  if (S > 1) {
    float *pk = a.part + ((static_cast<size_t>(blockIdx.x) * 2 + (SIDE ? 0 : 1)) * kOwn + (32 * kt + lrow)) * DH + 4 * half;
#pragma unroll
    for (int j = 0; j < K::kDT; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t x = {acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
        *reinterpret_cast<f32x4_t *>(pk + 32 * j + 8 * g) = x;
      }
    return;
  }
  if (kr >= T) return;
  bf16_t *out = static_cast<bf16_t *>(SIDE ? a.dk : a.dv) +
                (tok + kr) * (SIDE ? a.dk_stride : a.dv_stride) + static_cast<size_t>(kvh) * DH + 4 * half;
  const float f = SIDE ? a.scale : 1.0f;
#pragma unroll
  for (int j = 0; j < K::kDT; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<uint2 *>(out + 32 * j + 8 * g) =
          make_uint2(pack_bf16x2(acc[j][4 * g] * f, acc[j][4 * g + 1] * f),
                     pack_bf16x2(acc[j][4 * g + 2] * f, acc[j][4 * g + 3] * f));
}

template <int DH>
__global__ __launch_bounds__(64 * 2 * kWg, 2) void attn_dkv(AttnBwdArgs a) {
  __shared__ DkvLds<DH> sh;
  const int w = uni(threadIdx.x >> 6), lane = threadIdx.x & 63;
  // both sides pass the same number of barriers
  if (w < kWg)
    dkv_side<DH, 0>(a, sh, w, lane);
  else
    dkv_side<DH, 1>(a, sh, w - kWg, lane);
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
size_t attn_bwd_stat_bytes(int B, int T, int Hq) { return static_cast<size_t>(B) * T * Hq * sizeof(float2); }
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
  attn_dkv<DH><<<static_cast<unsigned>(a.slots) * a.B * a.Hkv, 64 * 2 * kWg, 0, s>>>(a);
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
