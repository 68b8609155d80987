// rglru_prefix.hip -- attention of one new token per sequence, the sequences sharing a prefix that the paged cache
// holds once (gfx950).
//
// Sequence n's tokens are the P of the prefix and then its own len[n]; token u < P lies where prefix_table says, own
// token j = u - P where block_table[n] says. Visible: u < L = P + len[n] and (u >= L - W or u < sinks).
//   o[n][h] = sum_u softmax_u(scale <q[n][h], K[u]>) V[u]
// A softmax over two sets of keys is joined from each set's maximum m, sum l and unnormalised O, so the prefix is read
// once for all sequences: their query heads on one key/value head are the rows of one product (this file's first
// kernel), each sequence's own tokens go through the paged decoding kernel (rglru_paged.hip), and the parts of both,
// each split over its length, are joined here.
//
// prefix_fwd: a workgroup has 128 rows (sequence, head of the group) and a chunk of the prefix, a wave 32 rows:
// S^T = K Q^T and O^T += V^T P^T on 32x32x16 MFMAs, a row per lane, P never leaving its lane, as in the prompt's
// attention (rglru_attn.h has the LDS layout). Blocks of 32 keys are in two LDS slots: bf16 rows go there directly,
// each lane with its row's address; e4m3 rows through registers, converted on the way with their scale (exact in
// bf16), so that both contractions see plain bf16 and one conversion serves 128 rows.
// A window may have left a part of the prefix for some rows and not for others: masked entries get P = 0, and where
// 0 * V is not 0 (a V that is infinite or NaN) the row is done again key by key.
//
// N256 Hq8 Hkv2 dh128 P32000 in e4m3, up to 400 own tokens: in a trace 71 us and 9.4 of joining, 73 in all timed among other
// passes. Matrix units are busy for 31% of the time (a third of it P's lower halves), vector units for 46% (a quarter of it the
// exponentials), and with the two or three waves that a SIMD's registers hold, the one hardly hides behind the other. The
// softmax of a block between the matrix instructions of the one before, or of all three stages, gained nothing (79 us for then
// 77, and 188, spilled).
// N64 Hq16 dh256 P1999 in bf16: 26 us and 6.4, most of it each chunk's latency and its O (17 MB); in e4m3 27 and 6.6, with 19
// registers spilled, 10 of which are read back in each block.
#include "rglru_attn.h"
#include "rglru_e4m3.h"
#include "rglru_grid.h"
#include "rglru_paged.h"

#include <algorithm>
#include <cmath>

namespace rglru {

using namespace attn;

namespace {

constexpr int kAhead = 2;  // MFMA steps that LDS operands are read ahead (3: 3% slower in e4m3 at dh128, else the same)

// dma_16b from an address per lane: 64 lanes x 16 bytes to LDS at lds_base + 16 lane.
__device__ __forceinline__ void dma_16b_from(const void *p, unsigned lds_base) {
  unsigned saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off\n\t"
      "s_nop 0\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(p), "s"(lds_base));
}

}  // namespace

// O (unnormalised), m and l of one row over the keys lo .. hi - 1, one key at a time (DH / 64 values per lane). Only
// for rows whose O came out non-finite although their sum is finite.
template <typename C, int DH>
__device__ __forceinline__ void prefix_row(const PrefixArgs &a, const bf16_t *q, int kvh, int lo, int hi, int w0,
                                           float *out, float *stat, int lane) {
  constexpr int kPer = DH / 64;
  float qv[kPer], o[kPer] = {};
#pragma unroll
  for (int i = 0; i < kPer; ++i) qv[i] = bf16_to_f32(q[lane * kPer + i]);
  float m = a.floor, l = 0.0f;
  for (int u = lo; u < hi; ++u) {
    if (u >= a.sinks && u < w0) {
      u = min(w0, hi) - 1;
      continue;
    }
    const int t = u / a.page, page = a.prefix_table[t];  // (a bad page makes the sum NaN: not done again)
    const size_t row = static_cast<size_t>(page) * a.page + (u - t * a.page), at = row * a.Hkv + kvh;
    float k[kPer], v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const size_t e = at * DH + lane * kPer + i;
      if constexpr (sizeof(C) == 2) {
        k[i] = bf16_to_f32(static_cast<const bf16_t *>(a.k_pages)[e]);
        v[i] = bf16_to_f32(static_cast<const bf16_t *>(a.v_pages)[e]);
      } else {
        k[i] = bf16lo(bf16x2_of<false>(static_cast<const uint8_t *>(a.k_pages)[e], 1.0f)) *
               scale_value(static_cast<const uint8_t *>(a.k_scales)[at]);
        v[i] = bf16lo(bf16x2_of<false>(static_cast<const uint8_t *>(a.v_pages)[e], 1.0f)) *
               scale_value(static_cast<const uint8_t *>(a.v_scales)[at]);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s = fmaf(qv[i], k[i], s);
#pragma unroll
    for (int e = 1; e < 64; e <<= 1) s += __shfl_xor(s, e, 64);
    const float mn = fmaxf(m, s);
    const float corr = __builtin_amdgcn_exp2f((m - mn) * a.c), p = __builtin_amdgcn_exp2f((s - mn) * a.c);
    m = mn;
    l = l * corr + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * corr + p * v[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) out[lane * kPer + i] = o[i];
  if (lane == 0) {
    stat[0] = m;
    stat[1] = l;
  }
}

constexpr unsigned kPartRow = 36 * 4;  // 32 values of a row on their way out, 16 bytes apart against conflicts

// What a workgroup of the prefix has in LDS: two blocks of K and V, then each wave's rows on their way out; each wave's
// first visible token; keys whose page is none, by block and wave.
template <int DH> struct PrefixLds {
  static constexpr unsigned kIn = 2 * Blk<DH>::kSlot, kOut = kOwn * kPartRow;
  __attribute__((aligned(1024))) unsigned char slots[kIn > kOut ? kIn : kOut];
  int least[kWg];
  unsigned bads[2][kWg];
};

// The prefix's part: id is the workgroup's (chunk, key/value head, 128 rows).
template <typename C, int DH>
__device__ __forceinline__ void prefix_rows(const PrefixArgs &a, int chunk, int id, PrefixLds<DH> &mem) {
  typedef Blk<DH> K;
  constexpr bool kCode = sizeof(C) == 1;
  auto &smem = mem.slots;
  auto &least = mem.least;
  auto &bads = mem.bads;
  const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6);
  const unsigned lds = lds_addr(smem);
  const int half = lane >> 5;
  const int G = a.Hq / a.Hkv;
  const long long R = static_cast<long long>(a.N) * G;  // rows of a key/value head
  const int tiles = static_cast<int>((R + kOwn - 1) / kOwn);
  // (row tiles first: the workgroups of one chunk are near each other)
  const int sp = uni(id / (tiles * a.Hkv)), rest = id - sp * tiles * a.Hkv;
  const int kvh = uni(rest / tiles), tile = rest - kvh * tiles;
  const int P = prefix_of(a.prefix_len, a.prefix_cap);
  const int blocks = (P + kBlk - 1) / kBlk, b0 = sp * chunk, b1 = min(blocks, b0 + chunk);
  if (b0 >= b1) return;  // (also without a prefix and with a bad length)
  // this lane's row
  struct Row {
    int n, h;
    bool on;     // is one
    size_t part;  // where its part goes
  };
  auto my_row = [&](int l) {
    const int r = tile * kOwn + 32 * w + (l & 31);  // (R is below 2^30)
    Row x;
    x.on = r < R;
    const int rc = x.on ? r : static_cast<int>(R) - 1;
    x.n = rc / G;
    x.h = kvh * G + rc - x.n * G;
    x.part = (static_cast<size_t>(x.n) * a.parts + sp) * a.Hq + x.h;
    return x;
  };
  int w0;  // tokens before it are behind the row's window (lens may be anything: the join refuses what is no length)
  bf16x8_t qf[K::kKS];
  {
    const Row x = my_row(lane);
    w0 = static_cast<int>(min(max(static_cast<long long>(P) + a.lens[x.n] - a.window, 0LL), 0x7FFFFFFFLL));
    const bf16_t *const q = static_cast<const bf16_t *>(a.q) + static_cast<size_t>(x.n) * a.q_stride +
                            static_cast<size_t>(x.h) * DH;
#pragma unroll
    for (int s = 0; s < K::kKS; ++s) qf[s] = load_bf16x8(q + 16 * s + 8 * half);
  }
  int wmin = w0, wmax = w0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    wmin = min(wmin, __shfl_xor(wmin, o, 64));
    wmax = max(wmax, __shfl_xor(wmax, o, 64));
  }
  wmin = uni(wmin);
  wmax = uni(wmax);
  if (lane == 0) least[w] = wmin;
  lds_barrier();
  const int first = min(min(least[0], least[1]), min(least[2], least[3]));
  // blocks that no row sees are left out: after the sinks' up to the first window's
  const int sink_end = (min(a.sinks, P) + kBlk - 1) / kBlk, win = first / kBlk;
  auto next_of = [&](int b) { return uni(b >= sink_end && b < win ? win : b); };
  const int i0 = next_of(b0);
  if (i0 >= b1) {  // nothing: l = 0, and O is not read
    const Row x = my_row(lane);
    if (half == 0 && x.on) {
      a.stat[2 * x.part] = a.floor;
      a.stat[2 * x.part + 1] = 0.0f;
    }
    return;
  }

  const unsigned row_bytes = static_cast<unsigned>(a.Hkv) * DH * sizeof(C);
  const char *const kp = static_cast<const char *>(a.k_pages) + static_cast<size_t>(kvh) * DH * sizeof(C);
  const char *const vp = static_cast<const char *>(a.v_pages) + static_cast<size_t>(kvh) * DH * sizeof(C);
  // A block's rows are looked up a block before they are loaded, and loaded a block before they are used. (What the
  // table gives is looked at when it is needed: at once, it would be waited for, and with it all loads before it.)
  // bf16: a lane looks up key lane % 32, and its row is handed to the lanes that load it.
  // e4m3: a thread has DH / 8 codes of key tid / 8.
  int key_page = 0, key_at = 0;  // of the key looked up, its page and place there
  constexpr int kCW = kCode ? DH / 32 : 1;  // words
  uint32_t ck[kCW], cv[kCW];
  unsigned sk = 0, sv = 0;
  // (the thread's terms are formed where they are needed: kept, they take registers from the walk)
  auto mine_of = [&]() {
    int x = threadIdx.x;
    asm volatile("" : "+v"(x));
    return x;
  };
  auto look_up = [&](int b) {
    const int u = min(b * kBlk + (kCode ? mine_of() >> 3 : mine_of() & 31), P - 1);  // (past the prefix: its last key)
    const int t = static_cast<int>(__umulhi(2u * u, a.page_factor) >> a.page_shift);  // u / page
    key_page = a.prefix_table[t];
    key_at = u - t * a.page;
  };
  auto bad_key = [&]() { return key_page < 0 || key_page >= a.num_pages; };
  auto key_row = [&]() { return bad_key() ? 0 : key_page * a.page + key_at; };  // the pool's; for a bad page row 0
  auto load_codes = [&]() {
    const int row = key_row();
    const char *const kr = kp + static_cast<size_t>(static_cast<unsigned>(row)) * row_bytes + (mine_of() & 7) * (DH / 8),
               *const vr = vp + (kr - kp);
#pragma unroll
    for (int i = 0; i < kCW; i += 4) {
      if constexpr (kCW >= 4) {
        const u32x4_t x = *reinterpret_cast<const u32x4_t *>(kr + 4 * i), y = *reinterpret_cast<const u32x4_t *>(vr + 4 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ck[(i + j) % kCW] = x[j];
          cv[(i + j) % kCW] = y[j];
        }
      } else {
        const u32x2_t x = *reinterpret_cast<const u32x2_t *>(kr), y = *reinterpret_cast<const u32x2_t *>(vr);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          ck[j % kCW] = x[j];
          cv[j % kCW] = y[j];
        }
      }
    }
    const size_t at = static_cast<size_t>(row) * a.Hkv + kvh;
    sk = static_cast<const uint8_t *>(a.k_scales)[at];
    sv = static_cast<const uint8_t *>(a.v_scales)[at];
  };
  auto put = [&](const uint32_t *codes, unsigned b, unsigned dst) {
    const float s = __uint_as_float(b << 23);
    const int me = mine_of(), crow = me >> 3, cpart = me & 7;
#pragma unroll
    for (int i = 0; i < kCW / 2; ++i) {  // a 16-byte chunk of 8 values
      u32x4_t v;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v[2 * j] = bf16x2_of<false>(codes[2 * i + j], s);
        v[2 * j + 1] = bf16x2_of<true>(codes[2 * i + j], s);
      }
      *(lds_u32x4_t *)static_cast<uintptr_t>(dst + crow * K::kRowBytes +
                                             (((cpart * (kCW / 2) + i) ^ K::swz(crow)) * 16)) = v;
    }
  };
  auto load_rows = [&](unsigned slot) {
    const int mine = key_row();
#pragma unroll
    for (int ii = 0; ii < K::kLPW; ++ii) {
      const int row = (w + kWg * ii) * K::kRPI + lane / K::kCPR;
      const size_t at = static_cast<size_t>(static_cast<unsigned>(__shfl(mine, row, 64))) * row_bytes +
                        static_cast<unsigned>(((lane % K::kCPR) ^ K::swz(row)) * 16);
      const unsigned dst = static_cast<unsigned>(uni(slot + (w + kWg * ii) * 1024));
      dma_16b_from(kp + at, dst);
      dma_16b_from(vp + at, static_cast<unsigned>(uni(dst + K::kBytes)));
    }
  };
  // bad keys of the block looked up last, bit by bit (e4m3: of the 8 that this wave looked up, for all waves)
  auto bad_bits = [&]() {
    const unsigned long long x = __ballot(bad_key());
    if constexpr (!kCode) return static_cast<unsigned>(x);
    unsigned bits = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) bits |= static_cast<unsigned>((x >> (8 * j)) & 1) << j;
    return bits << (8 * w);
  };

  const unsigned row_lane = K::row_lane(lane), col_lane = K::col_lane(lane);
  f32x16_t acc[K::kDT];  // O^T
#pragma unroll
  for (int j = 0; j < K::kDT; ++j) acc[j] = f32x16_t{};
  float m = a.floor, mc = m * a.c, l = 0.0f;
  int b = i0, bn = next_of(i0 + 1);  // this block and the next one
  look_up(b);
  unsigned bad_now = bad_bits(), bad_next = 0;
  if constexpr (kCode) {
    load_codes();
    if (bn < b1) look_up(bn);
    if (lane == 0) bads[0][w] = bad_now;
    put(ck, sk, lds);
    put(cv, sv, lds + K::kBytes);
    if (bn < b1) {
      load_codes();
      bad_next = bad_bits();
      if (next_of(bn + 1) < b1) look_up(next_of(bn + 1));
    }
  } else {
    load_rows(lds);
    if (bn < b1) look_up(bn);
  }
  for (int i = 0; b < b1; ++i) {
    const unsigned slot = lds + (i & 1) * K::kSlot, other = lds + (~i & 1) * K::kSlot;
    const int after = next_of(bn + 1);
    unsigned bad;
    if constexpr (kCode) {
      lds_barrier();  // block i is in its slot; everyone is done with block i - 1
      bad = bads[i & 1][0] | bads[i & 1][1] | bads[i & 1][2] | bads[i & 1][3];
      if (bn < b1) {
        if (lane == 0) bads[~i & 1][w] = bad_next;
        put(ck, sk, other);
        put(cv, sv, other + K::kBytes);
        if (after < b1) {
          load_codes();
          bad_next = bad_bits();
          const int then = next_of(after + 1);
          if (then < b1) look_up(then);
        }
      }
    } else {
      bad = bad_now;
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's rows of block i landed
      lds_barrier();                        // everyone's landed; everyone is done with block i - 1
      if (bn < b1) {
        load_rows(other);
        bad_now = bad_bits();
        if (after < b1) look_up(after);
      }
    }
    const int U = b * kBlk;
    b = bn;
    bn = after;
    if (U >= a.sinks && U + kBlk <= wmin) continue;  // this wave's rows see nothing of it
    // ---- S^T
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
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kr[d % (kAhead + 1)], qf[d], s, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    const bool full = U + kBlk <= P && (U >= wmax || U + kBlk <= a.sinks) && bad == 0;
    if (!full) {
      const int first = 4 * ((mine_of() >> 5) & 1);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int k = 8 * (e >> 2) + first + (e & 3), u = U + k;
        const bool on = u < P && (u >= w0 || u < a.sinks);
        s[e] = !on ? -__builtin_inff() : (bad >> k) & 1 ? __builtin_nanf("") : s[e];
      }
    }
    // ---- running softmax, the maximum raised only when it grows by more than 2^8
    float mx = fmaxf(s[0], s[1]), my = fmaxf(s[2], s[3]);
#pragma unroll
    for (int e = 4; e < 16; e += 2) {
      mx = fmaxf(mx, s[e]);
      my = fmaxf(my, s[e + 1]);
    }
    float lo, hi;
    halves(fmaxf(mx, my), lo, hi);
    mx = fmaxf(fmaxf(lo, hi), a.floor);
    const bool raise = (mx - m) * a.c > 8.0f;
    if (__any(raise)) {
      const float corr = raise ? __builtin_amdgcn_exp2f(mc - mx * a.c) : 1.0f;
      l *= corr;
      m = raise ? mx : m;
      mc = m * a.c;
#pragma unroll
      for (int j = 0; j < K::kDT; ++j) acc[j] *= corr;
    }
    // (s - m) c as one operation: m c is off by 2^-24 of itself, for all keys of a row alike, which o is not changed by;
    // between a row's parts, and before and after the maximum is raised, weights are off by as much
    u32x4_t p[2], pl[2];  // P of two 16-key steps as bf16 hi + lo
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float x = __builtin_amdgcn_exp2f(fmaf(s[e], a.c, -mc)), y = __builtin_amdgcn_exp2f(fmaf(s[e + 1], a.c, -mc));
      l += x + y;
      uint32_t hw = pack_bf16x2(x, y);
      asm("" : "+v"(hw));  // (else x is rounded a second time for the difference)
      p[e >> 3][(e >> 1) & 3] = hw;
      pl[e >> 3][(e >> 1) & 3] = pack_bf16x2(x - bf16lo(hw), y - bf16hi(hw));
    }
    // ---- O^T += V^T P^T
    {
      unsigned vs = slot + K::kBytes + col_lane;
      asm volatile("" : "+v"(vs));
      auto v_of = [&](int k) { return K::cols(vs, k & 1, k >> 1); };
      bf16x8_t vt[kAhead + 1];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) vt[k] = v_of(k);
#pragma unroll
      for (int k = 0; k < 2 * K::kDT; ++k) {
        if (k + kAhead < 2 * K::kDT) vt[(k + kAhead) % (kAhead + 1)] = v_of(k + kAhead);
        f32x16_t &o = acc[k >> 1];
        o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vt[k % (kAhead + 1)], __builtin_bit_cast(bf16x8_t, p[k & 1]), o, 0,
                                                    0, 0);
        o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vt[k % (kAhead + 1)], __builtin_bit_cast(bf16x8_t, pl[k & 1]), o, 0,
                                                    0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // ---- the part: lane = row, accumulator e of tile j is d = 32 j + 8 (e / 4) + 4 half + e % 4
  float lo, hi;
  halves(l, lo, hi);
  const float lt = lo + hi;
  float worst = 0.0f;
  int again = lane;
  asm volatile("" : "+v"(again));  // the row is formed anew: kept, it takes registers from the walk
  const Row me = my_row(again);
  // through LDS, 32 values of the wave's 32 rows at a time: whole lines to memory (lane by lane, 32 bytes of each)
  lds_barrier();  // everyone is done with the slots
  const unsigned mine = lds + w * 32 * kPartRow;
  const int sub = again >> 3;  // this lane stores 16 bytes of rows sub, 8 + sub, ..
  const size_t at = me.on ? me.part : static_cast<size_t>(-1);
  float *to[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long part = __shfl(static_cast<long long>(at), 8 * k + sub, 64);
    to[k] = part < 0 ? nullptr : a.part + part * DH + 4 * (again & 7);
  }
#pragma unroll
  for (int j = 0; j < K::kDT; ++j) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      u32x4_t x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        worst = fmaf(0.0f, acc[j][4 * g + e], worst);  // NaN if any is not finite
        x[e] = __float_as_uint(acc[j][4 * g + e]);
      }
      *(lds_u32x4_t *)static_cast<uintptr_t>(mine + (again & 31) * kPartRow + 32 * g + 16 * half) = x;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const u32x4_t x = *(lds_u32x4_t *)static_cast<uintptr_t>(mine + (8 * k + sub) * kPartRow + 16 * (again & 7));
      if (to[k]) *reinterpret_cast<u32x4_t *>(to[k] + 32 * j) = x;
    }
  }
  if (half == 0 && me.on) {
    a.stat[2 * me.part] = m;
    a.stat[2 * me.part + 1] = lt;
  }
  const unsigned long long rows = __ballot(me.on && !(worst == 0.0f) && lt < __builtin_inff());
  unsigned odd = static_cast<unsigned>(rows | (rows >> 32));
  if (odd) __builtin_amdgcn_s_waitcnt(0x0F70);  // this wave's stores are done before it stores those rows again
  while (odd) {
    const int x = __builtin_ctz(odd);
    odd &= odd - 1;
    const Row y = my_row(x);
    prefix_row<C, DH>(a, static_cast<const bf16_t *>(a.q) + static_cast<size_t>(y.n) * a.q_stride +
                             static_cast<size_t>(y.h) * DH,
                      kvh, b0 * kBlk, min(P, b1 * kBlk), __shfl(w0, x, 64), a.part + y.part * DH, a.stat + 2 * y.part, lane);
  }
}

// Both parts in one launch, the prefix's workgroups first: those are bound by their products and the vector work
// between them, the own tokens' by memory, and those fill the CUs that the longer ones leave.
// Three workgroups a CU at dh 128 (at dh 64 four): the prefix's are two, so that own tokens run beside them.
template <typename C, int DH, bool UNI>
__global__ __launch_bounds__(64 * kWg, DH == 128 ? 3 : 2) void prefix_fwd(PrefixArgs a, PagedArgs own, int chunk, int own_chunk, int own_splits,
                                                          int shared_groups, int own_groups) {
  __shared__ union Both {
    __device__ Both() {}
    PrefixLds<DH> prefix;
    PagedLds<DH> paged;
  } lds;
  const int id = block_of(blockIdx.y);
  const bool mine = id >= shared_groups;
  const int i = mine ? id - shared_groups : id;
  if (mine && i >= own_groups) return;
  if (mine) {
    const int cols = own.N * own_splits, y = i / cols;
    paged_rows<bf16_t, C, DH, UNI, true>(own, own_chunk, own_splits, i - y * cols, y, lds.paged);
  } else {
    prefix_rows<C, DH>(a, chunk, i, lds.prefix);
  }
}

// Joins a row's parts, those of the prefix and its own: workgroup = (row, head), a wave takes every fourth part.
template <int DH>
__global__ __launch_bounds__(256) void prefix_join(PrefixArgs a, PagedArgs own, int chunk, int own_chunk) {
  constexpr int V = DH / 64;
  __shared__ float ro[4][DH], rl[4], rm[4];
  const long long id = static_cast<long long>(block_of(blockIdx.y));
  if (id >= static_cast<long long>(a.N) * a.Hq) return;
  const int n = static_cast<int>(id / a.Hq), h = static_cast<int>(id - static_cast<long long>(n) * a.Hq);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int P = prefix_of(a.prefix_len, a.prefix_cap);
  const int raw = uniform_load(a.lens, n);
  const bool bad = P < 0 || raw < 0 || raw > static_cast<long long>(own.max_pages) * own.page;
  const Walk wk = walk_of<kBlk>(bad ? 0 : raw, a.window, max(0, a.sinks - P));
  const int shared = bad ? 0 : ((P + kBlk - 1) / kBlk + chunk - 1) / chunk;
  const int used = shared + (wk.nt + own_chunk - 1) / own_chunk;
  float m = a.floor, l = 0.0f, acc[V] = {};
  constexpr int kAt = 4;  // parts in flight
  for (int s0 = w; s0 < used; s0 += 4 * kAt) {
    float2 st[kAt];
    float x[kAt][V];
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      const int s = min(s0 + 4 * j, used - 1);
      const size_t r = (static_cast<size_t>(n) * a.parts + (s < shared ? s : own.first_part + s - shared)) * a.Hq + h;
      st[j] = *reinterpret_cast<const float2 *>(a.stat + 2 * r);
#pragma unroll
      for (int i = 0; i < V; ++i) x[j][i] = a.part[r * DH + lane * V + i];
    }
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      // (l = 0: the row sees nothing there, and O may hold anything)
      if (s0 + 4 * j >= used || st[j].y == 0.0f) continue;
      const float mn = fmaxf(m, st[j].x);
      const float fo = __builtin_amdgcn_exp2f((m - mn) * a.c), fn = __builtin_amdgcn_exp2f((st[j].x - mn) * a.c);
      m = mn;
      l = fmaf(st[j].y, fn, l * fo);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(x[j][i], fn, acc[i] * fo);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) ro[w][lane * V + i] = acc[i];
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
    o = bad ? __builtin_nanf("") : (P | raw) == 0 ? 0.0f : o / lt;
    static_cast<bf16_t *>(a.o)[static_cast<size_t>(id) * DH + d] = f32_to_bf16(o);
  }
}

// Blocks per chunk of the prefix, and the most chunks it can have. A chunk's length is time in which other CUs wait, and
// each chunk leaves an O of all rows to write and read again: short chunks suit few blocks and few row tiles, and the best
// length grows as the root of both (us at dh 256 in bf16, Hq16 Hkv1, with chunks of 1, 2, 4 and 8 blocks; other types and dh
// turn at the same places: 10 blocks of 1 tile 13.4 14.7 16.9 22.8, of 8 tiles 19.4 17.5 19.0 24.8; 63 of 1 tile 18.5 17.2
// 18.0 23.2, of 4 27.3 22.4 21.9 25.0; 250 of 1 tile 34.3 26.8 23.0 25.8, of 6 41.7 41.7 34.7 29.7). From 512 workgroups on,
// two a CU, chunks grow with the blocks.
PagedPlan prefix_plan(int N, int Hq, int Hkv, long long cap) {
  const long long tiles = (static_cast<long long>(N) * (Hq / Hkv) + kOwn - 1) / kOwn * Hkv;
  const long long blocks = (cap + kBlk - 1) / kBlk, all = blocks * tiles;
  constexpr long long kTarget = 512;  // workgroups: two fit a CU at a time
  const long long root = std::llround(std::sqrt(static_cast<double>(all)) / 5);
  const long long chunk = std::max((all + kTarget - 1) / kTarget, std::min<long long>(std::max<long long>(root, 1), 8));
  PagedPlan p;
  p.chunk = static_cast<int>(std::min<long long>(chunk, 1 << 28));
  p.splits = static_cast<int>(std::max<long long>((blocks + p.chunk - 1) / p.chunk, 1));
  return p;
}

namespace {

template <typename C, int DH>
hipError_t launch(const PrefixArgs &a, const PagedArgs &own, const PagedPlan &p, const PagedPlan &po, hipStream_t s) {
  const int G = a.Hq / a.Hkv;
  const long long tiles = (static_cast<long long>(a.N) * G + kOwn - 1) / kOwn;
  const long long shared = tiles * a.Hkv * p.splits;
  const long long mine = static_cast<long long>(a.N) * po.splits * a.Hkv * ((G + 15) / 16), all = shared + mine;
  const dim3 grid(grid_x(all), grid_rows(all));
  if (a.page % 16 == 0)
    prefix_fwd<C, DH, true><<<grid, 64 * kWg, 0, s>>>(a, own, p.chunk, po.chunk, po.splits, static_cast<int>(shared),
                                                      static_cast<int>(mine));
  else
    prefix_fwd<C, DH, false><<<grid, 64 * kWg, 0, s>>>(a, own, p.chunk, po.chunk, po.splits, static_cast<int>(shared),
                                                       static_cast<int>(mine));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const long long rows = static_cast<long long>(a.N) * a.Hq;
  prefix_join<DH><<<dim3(grid_x(rows), grid_rows(rows)), 256, 0, s>>>(a, own, p.chunk, po.chunk);
  return hipGetLastError();
}

template <typename C>
hipError_t launch(const PrefixArgs &a, const PagedArgs &own, const PagedPlan &p, const PagedPlan &po, hipStream_t s) {
  switch (own.dh) {
    case 64: return launch<C, 64>(a, own, p, po, s);
    case 128: return launch<C, 128>(a, own, p, po, s);
    case 256: return launch<C, 256>(a, own, p, po, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_prefix_attention(PrefixArgs a, const PagedArgs &own, const PagedPlan &p, const PagedPlan &po,
                                   hipStream_t s) {
  // u / page for u < 2^31 as (u f) >> (31 + s): 2^(s - 1) < page <= 2^s and f = floor(2^(31 + s) / page) + 1, which fits
  // 32 bits; f page - 2^(31 + s) is at most page, so u times it stays below 2^(31 + s)
  while ((1LL << a.page_shift) < a.page) ++a.page_shift;
  a.page_factor = static_cast<unsigned>((1ULL << (31 + a.page_shift)) / a.page + 1);
  return a.k_scales ? launch<uint8_t>(a, own, p, po, s) : launch<bf16_t>(a, own, p, po, s);
}

}  // namespace rglru
