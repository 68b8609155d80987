// rglru_mqa_bwd.hip -- gradients of local attention (rglru_local_attention), bf16 on gfx950.
//
// With s = q k^T, p = exp(scale s - lse) on the visible pairs (0 elsewhere), and given do = dL/do:
//   delta_t = <do_t, o_t>,  dp = do v^T,  ds = p (dp - delta),
//   dq = scale ds k,  dk = scale sum_heads ds^T q,  dv = sum_heads p^T do.
//
// Two kernels, each recomputing p, with no floating-point atomics (bitwise reproducible):
//   attn_dq   owns 128 rows of one query head and walks the key blocks they see; q and do are in registers,
//             K and V blocks in LDS: S^T = K Q^T, dP^T = V dO^T, dQ^T += K^T dS^T. It also forms delta.
//   attn_dkv  owns 128 keys and walks the (head of the group, block of 32 rows) items that see them; k and v
//             are in registers, Q and dO blocks in LDS: S = Q K^T, dP = dO V^T, dV^T += dO^T P,
//             dK^T += Q^T dS.
// In both, the accumulator layout of S and dP (one column per lane, 16 rows) is already the B operand's of the
// products that follow, if these take their k index in the accumulator's order, and the other operand of those
// products is a transpose of a block in LDS, read by ds_read_b64_tr_b16.
//
// The work of 32 rows (keys) is given to two waves of one SIMD, one for S and P, one for dP and dS: held by
// one wave, the operands and sums of both take the SIMD to itself, and nothing runs beside its exponentials.
// P goes from one to the other through LDS; products with it are a step behind, so that one barrier per step is
// enough and they fill the gaps between the dependent steps of S. (dq with one wave for both: 220 us where this
// takes 160 at B4 T2048 Hq10 dh256 W1024.)
//
// attn_dkv's items (rglru_shares.h) are dealt out in equal shares, one per CU, as the blocks' own numbers
// differ (the last keys of a sequence are seen by few rows, padded sequences have fewer, sinks are seen by all):
// 152-168 us instead of 190-202 with the same number of workgroups for every block, at the same sizes. Blocks that
// several workgroups share are summed by attn_dkv_sum, in order, from fp32 parts that lie in the accumulators'
// order (15 us; 256 shares: with 512, 27 us, and 172-180 us for attn_dkv).
#include "rglru_attn.h"
#include "rglru_grid.h"
#include "rglru_launch.h"
#include "rglru_shares.h"

#include <algorithm>
#include <type_traits>

namespace rglru {

using namespace attn;

namespace {

constexpr int kSlots = 3;      // blocks in LDS: the last one, this one, the next on its way
constexpr int kFewKeys = 256;  // rows with fewer keys: delta from the sums, not from o

// One block's products: returns R x, R the block's rows at `at` (kKS steps over d), and adds the block at
// `pt`, transposed, times pd into acc (as many steps: two 16-row steps for each 32-wide d tile). The two
// alternate, as the steps of R x wait for each other. Operands are read kAhead steps before their use:
// without that each MFMA waits for its own read.
template <int DH, bool kRows, bool kCols>
__device__ __forceinline__ f32x16_t products(unsigned at, unsigned pt, const bf16x8_t (&x)[Blk<DH>::kKS],
                                             const u32x4_t (&pd)[2], f32x16_t (&acc)[Blk<DH>::kDT]) {
  typedef Blk<DH> K;
  static_assert(2 * K::kDT == K::kKS, "as many steps of each");
  constexpr int kAhead = kRows && kCols ? 2 : 4;
  bf16x8_t r[kAhead], c[kAhead];
  f32x16_t s = f32x16_t{};
  asm volatile("" : "+v"(at), "+v"(pt));  // one register each; the steps' XORs are then with literals
  auto read = [&](int i) {
    if constexpr (kRows) r[i % kAhead] = K::rows(at, i);
    if constexpr (kCols) c[i % kAhead] = K::cols(pt, i & 1, i >> 1);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) read(i);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < K::kKS; ++i) {
    if constexpr (kRows) s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(r[i % kAhead], x[i], s, 0, 0, 0);
    if constexpr (kCols)
      acc[i >> 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          c[i % kAhead], __builtin_bit_cast(bf16x8_t, pd[i & 1]), acc[i >> 1], 0, 0, 0);
    if (i + kAhead < K::kKS) read(i + kAhead);
    __builtin_amdgcn_sched_barrier(0);
  }
  return s;
}

}  // namespace

// Workgroup = 128 rows of one query head, 8 waves: wave (rt, side) has rows 32 rt.. . Side 0 holds q, side 1
// do (B operands), so that two waves, one of each side, share a SIMD:
//   step i, side 0: S^T(i) = K Q^T, P(i) = exp2(c S - lse), handed over through LDS
//   step i, side 1: dP^T(i) = V dO^T; dS(i - 1) = P(i - 1) (dP(i - 1) - delta); dQ^T += K^T dS(i - 1)
template <int DH> struct DqLds {
  __attribute__((aligned(1024))) unsigned char blocks[kSlots * Blk<DH>::kSlot];
  f32x4_t px[2][kWg][4][64];  // P on its way to side 1
};

template <int DH, int SIDE>
__device__ __forceinline__ void dq_side(const AttnBwdArgs &a, DqLds<DH> &sh, int id, int rt, int lane) {
  typedef Blk<DH> K;
  const unsigned lds = lds_addr(sh.blocks);
  const int lrow = lane & 31, half = lane >> 5;
  const int T = a.T, Hq = a.Hq, W = a.window, sinks = a.sinks;
  // heavy first: query blocks from the last one down, all (sequence, head) pairs of one together
  const int nbh = a.B * Hq;
  const int nqb = (T + kOwn - 1) / kOwn;
  const int qi = uni(id / nbh), bh = id - qi * nbh;
  const int q0 = (nqb - 1 - qi) * kOwn;
  const int b = uni(bh / Hq), h = bh - b * Hq;
  const int len = clamp_len(a.lens, b, T);
  const int qw = q0 + 32 * rt, qr = qw + lrow;
  const size_t tok = static_cast<size_t>(b) * T;
  // what attn_dkv reads of the row: side 0 gives lse in exp2 units, side 1 delta
  const size_t sr = (static_cast<size_t>(b) * Hq + h) * T + min(qr, T - 1);
  bf16_t *const dq_ = static_cast<bf16_t *>(a.dq) + (tok + qw) * a.dq_stride + static_cast<size_t>(h) * DH;
  if (q0 >= len) {  // no row here reaches attn_dkv
    if (SIDE == 1)
#pragma unroll
      for (int p = 0; p < Tile<DH>::kPasses; ++p) {
        const int r = Tile<DH>::row(p, lane);
        if (qw + r < T)
          *reinterpret_cast<u32x4_t *>(dq_ + r * static_cast<size_t>(a.dq_stride) + 8 * (lane % K::kCPR)) = u32x4_t{};
      }
    return;
  }
  // this lane's row: q or do as B operand; side 1: delta = <do, o>
  bf16x8_t xf[K::kKS];
  float dl = 0.0f;
  const unsigned tile = lds + (SIDE * kWg + rt) * K::kBytes;  // this wave's, before the walk
  static_assert(sizeof(DqLds<DH>) >= 2 * kWg * K::kBytes, "a tile for each wave");
  {
    typedef Tile<DH> L;
    u32x4_t on[L::kPasses];
    if constexpr (SIDE == 1)
#pragma unroll
      for (int p = 0; p < L::kPasses; ++p)
        on[p] = *reinterpret_cast<const u32x4_t *>(
            static_cast<const bf16_t *>(a.o) +
            ((tok + min(qw + L::row(p, lane), T - 1)) * Hq + h) * DH + 8 * (lane % K::kCPR));
    const size_t xs = SIDE ? static_cast<size_t>(Hq) * DH : static_cast<size_t>(a.q_stride);
    L::start(static_cast<const bf16_t *>(SIDE ? a.do_ : a.q) + (tok + qw) * xs + static_cast<size_t>(h) * DH,
             static_cast<unsigned>(xs) * 2, len - qw, lane, tile);
    L::landed();
#pragma unroll
    for (int s = 0; s < K::kKS; ++s) xf[s] = L::operand(tile, lane, s);
    if constexpr (SIDE == 1) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int p = 0; p < L::kPasses; ++p)
        *(lds_u32x4_t *)static_cast<uintptr_t>(L::at(tile, p, lane)) = on[p];
      asm volatile("" ::: "memory");
#pragma unroll
      for (int s = 0; s < K::kKS; ++s) {
        const u32x4_t g = __builtin_bit_cast(u32x4_t, xf[s]);
        const u32x4_t o = __builtin_bit_cast(u32x4_t, L::operand(tile, lane, s));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dl = fmaf(bf16lo(g[e]), bf16lo(o[e]), fmaf(bf16hi(g[e]), bf16hi(o[e]), dl));
      }
      dl += __shfl_xor(dl, 32, 64);
    }
  }
  const bool in = qr < len;
  float l2 = 0.0f;
  if constexpr (SIDE == 0) {
    l2 = in ? a.lse[sr] * kLn2Inv : __builtin_inff();
    if (half == 0 && qr < T) a.lse2[sr] = l2;
  }
  asm volatile("" ::"v"(l2));  // complete its load here: the compiler does not see the loads that share its counter
  lds_barrier();               // everyone has its rows: the slots may be filled

  // side 0 brings the K rows, side 1 the V rows
  const BlockWalk walk_(q0, kOwn, len, W, sinks);
  const int n = walk_.n;
  const size_t stride = SIDE ? a.v_stride : a.k_stride;
  const unsigned rb = static_cast<unsigned>(stride) * 2;
  const bf16_t *const rows_ = static_cast<const bf16_t *>(SIDE ? a.v : a.k) + tok * stride +
                              static_cast<size_t>(uni(h / a.group)) * DH;
  const typename K::Lane ll = K::load_lane(rt, lane, rb);
  auto load_block = [&](int i, int sl) {
    const int u0 = walk_.first_row(i);
    const __amdgpu_buffer_rsrc_t src = K::rsrc(rows_ + static_cast<size_t>(u0) * stride, rb, len - u0);
#pragma unroll
    for (int ii = 0; ii < K::kLPW; ++ii)
      K::load(src, rb, ii, rt, ll, lds + sl * K::kSlot + (SIDE ? K::kBytes : 0u));
  };
  const unsigned row_lane = K::row_lane(lane) + (SIDE ? K::kBytes : 0u), col_lane = K::col_lane(lane);
  f32x16_t acc[K::kDT];  // side 1: dQ^T
  const bool none = (W == 1 && sinks == 0) || qr == 0;  // a row with one key has no gradient
  float sum_p = 0.0f, sum_pd = 0.0f;
  // one walk over the blocks; kDelta: only the sums of p dp and of p
  auto walk = [&](auto delta_only) {
    constexpr bool kDelta = decltype(delta_only)::value;
    u32x4_t pd[2] = {};         // side 1: dS of the last block
    if constexpr (SIDE == 1 && !kDelta)
#pragma unroll
      for (int j = 0; j < K::kDT; ++j) acc[j] = f32x16_t{};
    f32x16_t dpl = f32x16_t{};  // and its dP
    auto cols_of = [&](int sl) { return lds + sl * K::kSlot + col_lane; };
    auto take_p = [&](int buf) {  // side 1, of the last block
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const f32x4_t p = sh.px[buf][rt][e4][lane];
        if constexpr (kDelta) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum_p += p[e];
            sum_pd = fmaf(p[e], dpl[4 * e4 + e], sum_pd);
          }
        } else {
          float d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = p[e] * (dpl[4 * e4 + e] - dl);
          pd[e4 >> 1][2 * (e4 & 1)] = none ? 0u : pack_bf16x2(d[0], d[1]);
          pd[e4 >> 1][2 * (e4 & 1) + 1] = none ? 0u : pack_bf16x2(d[2], d[3]);
        }
      }
    };
    int sl = 0, slp = 0;  // slots of this block and the last (the first one: its own, with dS = 0)
    load_block(0, 0);
    for (int i = 0; i < n; ++i) {
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's rows of block i landed
      lds_barrier();  // everyone's landed, everyone is done with block i - 2 and P(i - 1) is written
      const int sln = sl == kSlots - 1 ? 0 : sl + 1;
      if (i + 1 < n) load_block(i + 1, sln);
      if constexpr (SIDE == 1)
        if (i > 0) take_p((i - 1) & 1);
      __builtin_amdgcn_sched_barrier(0);  // else reads of the steps below are moved up, past the registers there are
      f32x16_t s = products<DH, true, SIDE == 1 && !kDelta>(lds + sl * K::kSlot + row_lane, cols_of(slp), xf, pd, acc);
      if constexpr (SIDE == 0) {
        const int U = walk_.first_row(i);
        const bool full = U + 31 <= qw && (U > qw + 31 - W || U + 31 < sinks);
        if (!full) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int u = U + 8 * (e >> 2) + 4 * half + (e & 3);
            s[e] = sees(qr, u, W, sinks) ? s[e] : -__builtin_inff();
          }
        }
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          f32x4_t p;
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = __builtin_amdgcn_exp2f(fmaf(s[4 * e4 + e], a.c, -l2));
          sh.px[i & 1][rt][e4][lane] = p;
        }
      } else {
        dpl = s;
      }
      slp = sl;
      sl = sln;
    }
    lds_barrier();  // P of the last block
    if constexpr (SIDE == 1) {
      take_p((n - 1) & 1);
      if constexpr (!kDelta) products<DH, false, true>(0, cols_of(slp), xf, pd, acc);
    }
  };
  // delta from the rounded o is off by a 2^-9th of its terms, which averages out over many keys but
  // not over few, where dp - delta is a small difference: row blocks with fewer than kFewKeys keys
  // in some row take it as sum p dp / sum p instead, in a walk of its own.
  if (min(q0 + 1, W) < kFewKeys) {
    walk(std::true_type{});
    if constexpr (SIDE == 1) {
      sum_p += __shfl_xor(sum_p, 32, 64);
      sum_pd += __shfl_xor(sum_pd, 32, 64);
      dl = sum_pd / sum_p;
    }
  }
  if (SIDE == 1 && half == 0 && qr < T) a.delta[sr] = in ? dl : 0.0f;
  walk(std::false_type{});
  lds_barrier();  // everyone is done with the slots
  if constexpr (SIDE == 1) {
    const float f = a.scale;
    Tile<DH>::store(
        lds + rt * K::kBytes, lane,
        [&](int j, int g) {
          const u32x2_t v = {pack_bf16x2(acc[j][4 * g] * f, acc[j][4 * g + 1] * f),
                             pack_bf16x2(acc[j][4 * g + 2] * f, acc[j][4 * g + 3] * f)};
          return in ? v : u32x2_t{};
        },
        dq_, a.dq_stride, T - qw);
  }
}

// One workgroup's work beside attn_dq: first[e], the items before entry e = (sequence, key block) of one
// key/value head (the last: all of them), and span, the first and last workgroup that have a block's items
// (-1: there are none).
__device__ __forceinline__ void plan_items(const AttnBwdArgs &a) {
  const int nkb = (a.T + kOwn - 1) / kOwn, n = a.B * nkb, lane = threadIdx.x & 63;
  if (threadIdx.x < 64) {
    long long before = 0;
    for (int e0 = 0; e0 < n; e0 += 64) {
      const int e = e0 + lane, b = min(e / nkb, a.B - 1);
      const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
      const long long own =
          e < n ? static_cast<long long>(row_blocks((e - b * nkb) * kOwn, len, a.window, a.sinks)) * a.group : 0;
      long long sum = own;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const long long x = __shfl_up(sum, d, 64);
        if (lane >= d) sum += x;
      }
      if (e < n) a.first[e] = before + sum - own;
      before += __shfl(sum, 63, 64);
    }
    if (lane == 0) a.first[n] = before;
  }
  __syncthreads();
  const long long per_head = a.first[n], total = per_head * a.Hkv;
  const int G = share_count(total, a.groups);
  for (long long i = threadIdx.x; i < static_cast<long long>(n) * a.Hkv; i += 64 * 2 * kWg) {
    const long long head = i / n;
    const int e = static_cast<int>(i - head * n);
    const long long from = a.first[e], to = a.first[e + 1];
    a.span[i] = from == to ? make_int2(-1, -1)
                           : make_int2(share_of(total, G, head * per_head + from),
                                       share_of(total, G, head * per_head + to - 1));
  }
}

template <int DH>
__global__ __launch_bounds__(64 * 2 * kWg, 2) void attn_dq(AttnBwdArgs a) {
  __shared__ DqLds<DH> sh;
  const int id = block_of(blockIdx.y), last = (a.T + kOwn - 1) / kOwn * a.B * a.Hq;
  if (id >= last) {
    if (id == last) plan_items(a);
    return;
  }
  const int w = uni(threadIdx.x >> 6), lane = threadIdx.x & 63;
  // both sides pass the same number of barriers
  if (w < kWg)
    dq_side<DH, 0>(a, sh, id, w, lane);
  else
    dq_side<DH, 1>(a, sh, id, w - kWg, lane);
}

// Workgroup = 128 keys, 8 waves: wave (kt, side) has keys 32 kt.. . Side 0 holds k (B operands) and
// accumulates dV, side 1 holds v and accumulates dK, so that each fits in 256 registers and two waves,
// one of each side, share a SIMD:
//   step i, side 0: S(i) = Q K^T, P(i) = exp2(c S - lse), handed over through LDS; dV^T += dO^T P(i - 1)
//   step i, side 1: dP(i) = dO V^T; dS(i - 1) = P(i - 1) (dP(i - 1) - delta); dK^T += Q^T dS(i - 1)
// Both hold the same elements of S and dP in a lane, so the exchange is 16 values per lane, written and
// read in the lane's own order, and the one-step lag makes one barrier per step enough.
template <int DH> struct DkvLds {
  __attribute__((aligned(1024))) unsigned char blocks[kSlots * Blk<DH>::kSlot];
  f32x4_t px[2][kWg][4][64];       // P on its way to side 1
  float rowv[2][kSlots][2 * kBlk]; // the rows' lse in exp2 units, their delta (and room for what a load writes)
};

template <int DH, int SIDE>
__device__ __forceinline__ void dkv_side(const AttnBwdArgs &a, DkvLds<DH> &sh, int kt, int lane_) {
  typedef Blk<DH> K;
  const unsigned lds = lds_addr(sh.blocks);
  const int T = a.T, Hq = a.Hq, W = a.window, sinks = a.sinks;
  const int nkb = (T + kOwn - 1) / kOwn, n = a.B * nkb;
  const long long per_head = uniform_load(a.first, n), total = per_head * a.Hkv;
  const int G = share_count(total, a.groups);
  if (static_cast<int>(blockIdx.x) >= G) return;  // (the whole workgroup)
  // neighbouring shares, which read the same rows, on one XCD
  const int wg = G % 8 ? blockIdx.x : blockIdx.x % 8 * (G / 8) + blockIdx.x / 8;
  const long long hi = uni64(share_lo(total, G, wg + 1));
  for (long long pos = uni64(share_lo(total, G, wg)); pos < hi;) {  // a key block's items, or some of them
    int lane = lane_;
    asm volatile("" : "+v"(lane));  // the lane's terms are formed anew: kept, they take registers
    const int lrow = lane & 31, half = lane >> 5;
    const int kvh = uni(static_cast<int>(pos / per_head));
    const long long in_head = pos - kvh * per_head;
    int e = 0;  // the entry: the last with first[e] <= in_head, 64 places at a time
    for (int end = n; end - e > 1;) {
      const int step = (end - e + 63) / 64, at = e + lane * step;
      const int c = __popcll(__ballot(at < end && a.first[min(at, n)] <= in_head));
      e = uni(e + (c - 1) * step);
      end = uni(min(end, e + step));
    }
    const long long from = uniform_load(a.first, e);
    const int items = uni(static_cast<int>(uniform_load(a.first, e + 1) - from));
    const int i0 = uni(static_cast<int>(in_head - from));
    const int i1 = uni(static_cast<int>(min(static_cast<long long>(items), i0 + hi - pos)));
    pos += i1 - i0;
    const int b = uni(e / nkb), kb = e - b * nkb;
    const int K0 = kb * kOwn;
    const int len = clamp_len(a.lens, b, T);
    const int kw = K0 + 32 * kt, kr = kw + lrow;
    const size_t tok = static_cast<size_t>(b) * T;
    // this lane's key: k or v as B operand (rows past the sequence: zero)
    bf16x8_t kf[K::kKS];
    {
      typedef Tile<DH> L;
      const unsigned tile = lds + (SIDE * kWg + kt) * K::kBytes;
      const size_t xs = static_cast<size_t>(SIDE ? a.v_stride : a.k_stride);
      L::start(static_cast<const bf16_t *>(SIDE ? a.v : a.k) + (tok + kw) * xs + static_cast<size_t>(kvh) * DH,
               static_cast<unsigned>(xs) * 2, len - kw, lane, tile);
      L::landed();
#pragma unroll
      for (int s = 0; s < K::kKS; ++s) kf[s] = L::operand(tile, lane, s);
      lds_barrier();  // everyone has its keys: the slots may be filled
    }
    f32x16_t acc[K::kDT];  // dV^T or dK^T
#pragma unroll
    for (int j = 0; j < K::kDT; ++j) acc[j] = f32x16_t{};
    const int qfirst = K0 / kBlk, nq = uni(items / a.group);
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
          wave_uniform((SIDE ? a.delta : a.lse2) + (static_cast<size_t>(b) * Hq + h) * T + q0),
          static_cast<short>(0), uni(min(len - q0, kBlk) * 4), kRawWord3);
      const __amdgpu_buffer_rsrc_t src =
          K::rsrc(rows_ + static_cast<size_t>(q0) * (rb / 2) + static_cast<size_t>(h) * DH, rb, len - q0);
#pragma unroll
      for (int ii = 0; ii < K::kLPW; ++ii)
        K::load(src, rb, ii, kt, ll, lds + sl * K::kSlot + (SIDE ? K::kBytes : 0u));
      dma_4b(st, lane * 4, lds_addr(sh.rowv[SIDE][sl]));
    };
    const unsigned row_lane = K::row_lane(lane) + (SIDE ? K::kBytes : 0u);  // side 0 reads Q, 1 dO
    const unsigned col_lane = K::col_lane(lane) + (SIDE ? 0u : K::kBytes);  // side 0 reads dO, 1 Q
    u32x4_t pd[2] = {};         // P (side 0) or dS (side 1) of the last item
    auto cols_of = [&](int sl) { return lds + sl * K::kSlot + col_lane; };
    f32x16_t dpl = f32x16_t{};  // side 1: dP of the last item
    // side 1: dS of the last item (first row Ql) from its P, dP and delta
    auto make_ds = [&](int buf, int sl, int Ql) {
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const f32x4_t p = sh.px[buf][kt][e4][lane];
        const f32x4_t dl = *reinterpret_cast<const f32x4_t *>(&sh.rowv[1][sl][8 * e4 + 4 * half]);
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = p[e] * (dpl[4 * e4 + e] - dl[e]);
        if (one) d[0] = d[1] = d[2] = d[3] = 0.0f;  // a row with one key has no gradient
        if (Ql + 8 * e4 + 4 * half == 0) d[0] = 0.0f;
        pd[e4 >> 1][2 * (e4 & 1)] = pack_bf16x2(d[0], d[1]);
        pd[e4 >> 1][2 * (e4 & 1) + 1] = pack_bf16x2(d[2], d[3]);
      }
    };
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
      f32x16_t s = products<DH, true, true>(lds + sl * K::kSlot + row_lane, cols_of(slp), kf, pd, acc);
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
          const f32x4_t l2 = *reinterpret_cast<const f32x4_t *>(&sh.rowv[0][sl][8 * e4 + 4 * half]);
          f32x4_t p;
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = __builtin_amdgcn_exp2f(fmaf(s[4 * e4 + e], a.c, -l2[e]));
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
    products<DH, false, true>(0, cols_of(slp), kf, pd, acc);
    lds_barrier();  // everyone is done with the slots
    if (i1 - i0 < items) {
      // a part: in the accumulators' order (attn_dkv_sum's units)
      float *const part = a.part + ((2 * static_cast<size_t>(wg) + (i0 == 0)) * 2 + SIDE) * kOwn * DH +
                          static_cast<size_t>(kt) * 32 * DH + 4 * lane;
#pragma unroll
      for (int j = 0; j < K::kDT; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<f32x4_t *>(part + (4 * j + g) * 256) =
              f32x4_t{acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
    } else {
      const float f = SIDE ? a.scale : 1.0f;
      const size_t os = static_cast<size_t>(SIDE ? a.dk_stride : a.dv_stride);
      Tile<DH>::store(
          lds + (SIDE * kWg + kt) * K::kBytes, lane,
          [&](int j, int g) {
            return u32x2_t{pack_bf16x2(acc[j][4 * g] * f, acc[j][4 * g + 1] * f),
                           pack_bf16x2(acc[j][4 * g + 2] * f, acc[j][4 * g + 3] * f)};
          },
          static_cast<bf16_t *>(SIDE ? a.dk : a.dv) + (tok + kw) * os + static_cast<size_t>(kvh) * DH, os, T - kw);
    }
  }
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

// dk, dv of the key blocks that several workgroups share: their parts in order; and zeros for the blocks
// without items. Grid: DH / 4 workgroups for each of span's entries; a lane has four values of a row.
template <int DH> __global__ __launch_bounds__(256) void attn_dkv_sum(AttnBwdArgs a) {
  constexpr int kPer = DH / 8;  // workgroups for dV, then as many for dK
  const int id = block_of(blockIdx.y), i = uni(id / (2 * kPer)), sub = id - i * 2 * kPer;
  const int nkb = (a.T + kOwn - 1) / kOwn, n = a.B * nkb;
  if (i >= n * a.Hkv) return;
  const int side = sub / kPer, unit = (sub - side * kPer) * 256 + threadIdx.x;  // of 32 DH
  const int2 span = {uniform_load(&a.span[i].x, 0), uniform_load(&a.span[i].y, 0)};
  if (span.x >= 0 && span.x == span.y) return;  // stored by attn_dkv
  f32x4_t acc = {};
  if (span.x >= 0) {
    const float *const part = a.part + static_cast<size_t>(side) * kOwn * DH + 4 * unit;
    constexpr int kAt = 4;  // parts whose loads are under way at a time
    for (int w0 = span.x; w0 <= span.y; w0 += kAt) {
      f32x4_t x[kAt];
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const int w = min(w0 + j, span.y);
        x[j] = *reinterpret_cast<const f32x4_t *>(part + (2 * static_cast<size_t>(w) + (w == span.x)) * 2 * kOwn * DH);
      }
#pragma unroll
      for (int j = 0; j < kAt; ++j)
        if (w0 + j <= span.y) acc += x[j];
    }
  }
  const int kvh = uni(i / n), e = i - kvh * n, b = uni(e / nkb), kb = e - b * nkb;
  const int kt = unit / (8 * DH), r = unit - kt * 8 * DH, lane = r & 63;  // r: (4 j + g) 64 + lane
  const int t = kb * kOwn + 32 * kt + (lane & 31);
  if (t >= a.T) return;
  const float f = side ? a.scale : 1.0f;
  bf16_t *const out = static_cast<bf16_t *>(side ? a.dk : a.dv) +
                      (static_cast<size_t>(b) * a.T + t) * (side ? a.dk_stride : a.dv_stride) +
                      static_cast<size_t>(kvh) * DH + 8 * (r >> 6) + 4 * (lane >> 5);
  *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f));
}

// One workgroup of attn_dkv per CU, fewer where its share would be below kMinShare items.
AttnBwdPlan attn_bwd_plan(int B, int T, int Hq, int Hkv, int window, int sinks) {
  constexpr long long kGroups = 256, kMinShare = 4;
  const long long nkb = (T + kOwn - 1) / kOwn, q_all = (T + kBlk - 1) / kBlk;
  const long long q_win = std::min<long long>(q_all, (kOwn + static_cast<long long>(window)) / kBlk + 1);
  const long long with_sinks = std::min<long long>((std::min(sinks, T) + kOwn - 1) / kOwn, nkb);
  const long long items = (with_sinks * q_all + (nkb - with_sinks) * q_win) * B * Hq;  // at most
  AttnBwdPlan p;
  p.entries = static_cast<size_t>(nkb) * B;
  p.groups = static_cast<int>(std::min<long long>(kGroups, std::max<long long>(1, items / kMinShare)));
  return p;
}

namespace {

template <int DH> hipError_t launch(const AttnBwdArgs &a, hipStream_t s) {
  const long long nq = (a.T + kOwn - 1) / kOwn, dq = nq * a.B * a.Hq + 1, sum = nq * a.B * a.Hkv * (DH / 4);
  attn_dq<DH><<<dim3(grid_x(dq), grid_rows(dq)), 64 * 2 * kWg, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  attn_dkv<DH><<<static_cast<unsigned>(a.groups), 64 * 2 * kWg, 0, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  attn_dkv_sum<DH><<<dim3(grid_x(sum), grid_rows(sum)), 256, 0, s>>>(a);
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
