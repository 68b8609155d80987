// rglru_shares.h -- how the key side of the local attention backward is divided: plain arithmetic, the same on the
// host (whose tests call it) and in the kernels.
//
// The work is a list of items: for each key/value head and each sequence's key blocks (in that order), the
// (head of the group, 32-row block) pairs that see some of the block's keys. Of n workgroups that take part,
// workgroup w has the items [share_lo(w), share_lo(w + 1)).
#pragma once

#ifdef __HIPCC__
#define RGLRU_HD __host__ __device__ __forceinline__
#else
#define RGLRU_HD inline
#endif

namespace rglru {
namespace attn {

constexpr int kWg = 4;          // waves (or pairs of waves) of a workgroup that own 32 rows or keys each
constexpr int kOwn = 32 * kWg;  // rows or keys per workgroup
constexpr int kBlk = 32;        // rows per LDS block

// Row blocks that see some of the keys K0 .. K0 + kOwn - 1 of a sequence of len tokens.
RGLRU_HD int row_blocks(int K0, int len, int window, int sinks) {
  if (K0 >= len) return 0;
  const long long behind = static_cast<long long>(K0) + kOwn - 2 + window;  // the last row whose window has one
  const int last = K0 < sinks || behind > len - 1 ? len - 1 : static_cast<int>(behind);
  return last / kBlk - K0 / kBlk + 1;
}

// Workgroups that take part. The launch's number comes from the sizes, the items from the lengths, which only
// the device knows: in a batch much shorter than T there are fewer items than workgroups. Then one item each, so that
// no share is empty: a block's parts are those of ALL workgroups from its first to its last.
RGLRU_HD int share_count(long long items, int groups) { return items < groups ? static_cast<int>(items) : groups; }

RGLRU_HD long long share_lo(long long items, int n, int w) { return items * w / n; }

// The workgroup that has item i: the largest w with share_lo(w) <= i.
RGLRU_HD int share_of(long long items, int n, long long i) { return static_cast<int>(((i + 1) * n - 1) / items); }

}  // namespace attn
}  // namespace rglru
