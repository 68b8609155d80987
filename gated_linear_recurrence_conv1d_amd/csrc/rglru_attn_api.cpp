// rglru_attn_api.cpp -- the C ABI of the local attention block's operators (include/rglru.h): argument
// checks and kernel launches. No allocation, no global state; every call is asynchronous on its
// stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "rglru.h"
#include "rglru_check.h"
#include "rglru_grid.h"
#include "rglru_launch.h"

namespace {

using rglru::aligned;
using rglru::check_heads;
using rglru::elem_bytes;
using rglru::flat;
using rglru::heads_of;
using rglru::hip_status;
using rglru::kBF16;
using rglru::kF32;
using rglru::kMaxStride;
using rglru::kMaxTokens;
using rglru::max_floor;
using rglru::overlaps;
using rglru::Rows;
using rglru::same;
using rglru::stride_ok;

rglru_status check_rope(int rows, int Hq, int Hkv, int dh, int rot, float eps, rglru_dtype dt,
                        const float *q_w, const float *k_w, const float *inv_freq) {
  const rglru_status st = check_heads(rows, Hq, Hkv, dh, dt);
  if (st != RGLRU_OK) return st;
  if (rot < 0 || rot > dh || rot % 2) return RGLRU_ERR_INVALID_ARG;
  if (dh % 2 || dh > rglru::kRopeMaxDh) return RGLRU_ERR_UNSUPPORTED;
  if ((q_w == nullptr) != (k_w == nullptr)) return RGLRU_ERR_INVALID_ARG;
  if (rot > 0 && !inv_freq) return RGLRU_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return RGLRU_ERR_INVALID_ARG;
  return RGLRU_OK;
}

rglru_status check_attn(int B, int T, int Hq, int Hkv, int dh, long long q_stride,
                        long long k_stride, long long v_stride, int window, int sinks, float scale,
                        rglru_dtype dt) {
  if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || dh < 1 || window < 1 || sinks < 0)
    return RGLRU_ERR_INVALID_ARG;
  if (Hq % Hkv) return RGLRU_ERR_INVALID_ARG;
  if (!(scale == scale) || scale < 0.0f || std::isinf(scale)) return RGLRU_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, Hq, dh) || !stride_ok(k_stride, Hkv, dh) || !stride_ok(v_stride, Hkv, dh))
    return RGLRU_ERR_INVALID_ARG;
  if (q_stride % 8 || k_stride % 8 || v_stride % 8) return RGLRU_ERR_INVALID_ARG;
  if (dt != RGLRU_BF16 || !rglru::local_mqa_supported(dh)) return RGLRU_ERR_UNSUPPORTED;
  if (B > 65535 || Hq > 65535) return RGLRU_ERR_UNSUPPORTED;
  if (q_stride > kMaxStride || k_stride > kMaxStride || v_stride > kMaxStride)
    return RGLRU_ERR_UNSUPPORTED;
  // workgroups of 128 rows, and one more in the backward
  if ((T + 127LL) / 128 * B * Hq >= rglru::kMaxBlocks) return RGLRU_ERR_UNSUPPORTED;
  // a sequence's k and v below 2 GiB: the sizes that are tested (the kernels' addresses are 64-bit down to a block
  // of 32 rows, whose offsets kMaxStride bounds)
  constexpr long long kRange = 1LL << 31;
  if (T * k_stride * 2 >= kRange || T * v_stride * 2 >= kRange) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

// The sum over workgroups' parts has dh / 4 workgroups for each key block.
bool bwd_grid_ok(int B, int T, int Hkv, int dh) {
  return (T + 127LL) / 128 * B * Hkv * (dh / 4) <= rglru::kMaxBlocks;
}

// Where the parts of the attention backward's workspace begin (lse2 first), and its size.
struct AttnBwdLayout {
  size_t delta, part, first, span, total;
};
AttnBwdLayout attn_bwd_layout(const rglru::AttnBwdPlan &p, int B, int T, int Hq, int Hkv, int dh) {
  using rglru::align_up;
  AttnBwdLayout l;
  l.delta = align_up(static_cast<size_t>(B) * T * Hq * sizeof(float));
  l.part = 2 * l.delta;
  // per workgroup: a block begun before its share and one that goes on behind it, dV and dK of 128 keys
  l.first = l.part + align_up(static_cast<size_t>(p.groups) * 2 * 2 * 128 * dh * sizeof(float));
  l.span = l.first + align_up((p.entries + 1) * sizeof(long long));
  l.total = l.span + align_up(p.entries * Hkv * sizeof(int2));
  return l;
}

rglru_status check_paged(int N, int Hq, int Hkv, int dh, int page_size, int max_pages, int window,
                         int sinks, rglru_dtype dt) {
  if (page_size < 1 || max_pages < 1 || window < 1 || sinks < 0) return RGLRU_ERR_INVALID_ARG;
  const rglru_status st = check_heads(N, Hq, Hkv, dh, dt);
  if (st != RGLRU_OK) return st;
  if (Hq % Hkv) return RGLRU_ERR_INVALID_ARG;
  if (!rglru::local_mqa_supported(dh)) return RGLRU_ERR_UNSUPPORTED;
  // one grid row per 16 heads of a group; one grid column per (sequence, chunk)
  if (static_cast<long long>(Hkv) * ((Hq / Hkv + 15) / 16) > 65535) return RGLRU_ERR_UNSUPPORTED;
  if (static_cast<long long>(N) * Hq > (1LL << 30)) return RGLRU_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size >= kMaxTokens) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

rglru::PagedPlan plan_of(int N, int Hq, int Hkv, int page_size, int max_pages, int window,
                         int sinks, rglru_dtype dt) {
  return rglru::paged_plan(N, Hq, Hkv, static_cast<long long>(max_pages) * page_size, window, sinks,
                           dt == RGLRU_BF16 ? kBF16 : kF32);
}

// The chunks' O, then their (m, l).
size_t paged_part_bytes(const rglru::PagedPlan &p, int N, int Hq, int dh) {
  return rglru::align_up(static_cast<size_t>(N) * p.splits * Hq * dh * sizeof(float));
}
size_t paged_bytes(const rglru::PagedPlan &p, int N, int Hq, int dh) {
  if (p.splits == 1) return 0;
  return paged_part_bytes(p, N, Hq, dh) +
         rglru::align_up(static_cast<size_t>(N) * p.splits * Hq * 2 * sizeof(float));
}

// What every attention over a paged cache asks of its tensors.
rglru_status check_paged_tensors(const void *q, const void *k_pages, const void *v_pages, const void *k_scales,
                                 const void *v_scales, const int *block_table, const int *lens, const void *o, int N,
                                 int Hq, int Hkv, int dh, long long q_stride, int num_pages, int page_size,
                                 int max_pages, float scale, rglru_dtype dt, const void *workspace,
                                 size_t workspace_bytes, size_t need) {
  if (num_pages < 1 || !(scale == scale) || scale < 0.0f || std::isinf(scale))
    return RGLRU_ERR_INVALID_ARG;
  if (static_cast<long long>(num_pages) * page_size >= kMaxTokens) return RGLRU_ERR_UNSUPPORTED;
  if (!q || !k_pages || !v_pages || !block_table || !lens || !o) return RGLRU_ERR_INVALID_ARG;
  const size_t e = elem_bytes(dt);
  if (!stride_ok(q_stride, Hq, dh) || q_stride * e % 16) return RGLRU_ERR_INVALID_ARG;
  const void *vec16[] = {q, k_pages, v_pages};
  for (const void *p : vec16)
    if (!aligned(p, 16)) return RGLRU_ERR_INVALID_ARG;
  if (!aligned(o, e) || !aligned(block_table, 4) || !aligned(lens, 4)) return RGLRU_ERR_INVALID_ARG;
  if (need && (!workspace || workspace_bytes < need)) return RGLRU_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return RGLRU_ERR_INVALID_ARG;
  const size_t heads = static_cast<size_t>(num_pages) * page_size * Hkv, pool = heads * dh * (k_scales ? 1 : e);
  const Rows outs[] = {flat(o, static_cast<size_t>(N) * Hq * dh * e),
                       flat(need ? workspace : nullptr, need)};
  const Rows ins[] = {heads_of(q, N, Hq, dh, q_stride, dt), flat(k_pages, pool), flat(v_pages, pool),
                      flat(k_scales, heads), flat(v_scales, heads),
                      flat(block_table, static_cast<size_t>(N) * max_pages * sizeof(int)),
                      flat(lens, static_cast<size_t>(N) * sizeof(int))};
  for (const Rows &w : outs)
    for (const Rows &r : ins)
      if (overlaps(w, r)) return RGLRU_ERR_INVALID_ARG;
  return overlaps(outs[0], outs[1]) ? RGLRU_ERR_INVALID_ARG : RGLRU_OK;
}

rglru_status paged_attention(const void *q, const void *k_pages, const void *v_pages, const void *k_scales,
                             const void *v_scales, const int *block_table, const int *lens, void *o, int N, int Hq,
                             int Hkv, int dh, long long q_stride, int num_pages, int page_size, int max_pages,
                             int window, int sinks, float scale, rglru_dtype dt, void *workspace,
                             size_t workspace_bytes, void *stream) {
  const rglru_status st = check_paged(N, Hq, Hkv, dh, page_size, max_pages, window, sinks, dt);
  if (st != RGLRU_OK) return st;
  const rglru::PagedPlan plan = plan_of(N, Hq, Hkv, page_size, max_pages, window, sinks, dt);
  const size_t need = paged_bytes(plan, N, Hq, dh);
  const rglru_status sp = check_paged_tensors(q, k_pages, v_pages, k_scales, v_scales, block_table, lens, o, N, Hq, Hkv,
                                              dh, q_stride, num_pages, page_size, max_pages, scale, dt, workspace,
                                              workspace_bytes, need);
  if (sp != RGLRU_OK) return sp;
  if (scale == 0.0f) scale = 1.0f / std::sqrt(static_cast<float>(dh));
  const float c = scale * 1.4426950408889634f;
  char *ws = static_cast<char *>(workspace);
  rglru::PagedArgs a = {q,        k_pages, v_pages, block_table, lens,      o,         nullptr,
                        nullptr,  N,       Hq,      Hkv,         dh,        q_stride,  num_pages,
                        page_size, max_pages, window, sinks,     c,         max_floor(c), k_scales,  v_scales,
                        nullptr,  0,       0,       0};
  if (need) {
    a.part = reinterpret_cast<float *>(ws);
    a.stat = reinterpret_cast<float *>(ws + paged_part_bytes(plan, N, Hq, dh));
  }
  (void)hipGetLastError();
  return hip_status(rglru::launch_paged_attention(a, plan, dt == RGLRU_BF16 ? kBF16 : kF32,
                                                  static_cast<hipStream_t>(stream)));
}

// Attention over a shared prefix: the own tokens' sizes as in paged attention, and the prefix's.
rglru_status check_prefix(int N, int Hq, int Hkv, int dh, int page_size, int prefix_pages, int max_pages, int window,
                          int sinks) {
  if (prefix_pages < 1) return RGLRU_ERR_INVALID_ARG;
  const rglru_status st = check_paged(N, Hq, Hkv, dh, page_size, max_pages, window, sinks, RGLRU_BF16);
  if (st != RGLRU_OK) return st;
  if (static_cast<long long>(prefix_pages) * page_size >= kMaxTokens) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}
struct PrefixPlans {
  rglru::PagedPlan shared, own;
  size_t part_bytes, bytes;
};
PrefixPlans prefix_plans(int N, int Hq, int Hkv, int dh, int page_size, int prefix_pages, int max_pages, int window,
                         int sinks) {
  PrefixPlans p;
  p.shared = rglru::prefix_plan(N, Hq, Hkv, static_cast<long long>(prefix_pages) * page_size);
  p.own = plan_of(N, Hq, Hkv, page_size, max_pages, window, sinks, RGLRU_BF16);
  const size_t rows = static_cast<size_t>(N) * (static_cast<size_t>(p.shared.splits) + p.own.splits) * Hq;
  p.part_bytes = rglru::align_up(rows * dh * sizeof(float));
  p.bytes = p.part_bytes + rglru::align_up(rows * 2 * sizeof(float));
  return p;
}

}  // namespace

extern "C" {

rglru_status rglru_qk_norm_rope(const void *q, const void *k, const void *v, const float *q_w,
                                const float *k_w, const float *inv_freq, const int *positions,
                                const long long *slots, void *q_out, void *k_out, void *k_pages,
                                void *v_pages, int rows, int Hq, int Hkv, int dh, int rot,
                                long long q_stride, long long k_stride, long long v_stride,
                                long long q_out_stride, long long k_out_stride, long long n_slots,
                                float eps, rglru_dtype dt, void *stream) {
  rglru_status st = check_rope(rows, Hq, Hkv, dh, rot, eps, dt, q_w, k_w, inv_freq);
  if (st != RGLRU_OK) return st;
  if (!q || !k || !positions || !q_out) return RGLRU_ERR_INVALID_ARG;
  if (slots ? (!v || !k_pages || !v_pages || n_slots < 1) : !k_out) return RGLRU_ERR_INVALID_ARG;
  if (!slots) {
    v = nullptr;
    k_pages = v_pages = nullptr;
    v_stride = n_slots = 0;
  }
  if (!k_out) k_out_stride = 0;
  if (!stride_ok(q_stride, Hq, dh) || !stride_ok(k_stride, Hkv, dh) ||
      !stride_ok(q_out_stride, Hq, dh) || (k_out && !stride_ok(k_out_stride, Hkv, dh)) ||
      (v && !stride_ok(v_stride, Hkv, dh)))
    return RGLRU_ERR_INVALID_ARG;
  const size_t e = elem_bytes(dt);
  const void *vec[] = {q, k, v, q_out, k_out, k_pages, v_pages};
  for (const void *p : vec)
    if (!aligned(p, e)) return RGLRU_ERR_INVALID_ARG;
  const void *vec4[] = {q_w, k_w, inv_freq, positions};
  for (const void *p : vec4)
    if (!aligned(p, 4)) return RGLRU_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return RGLRU_ERR_INVALID_ARG;
  const Rows rq = heads_of(q, rows, Hq, dh, q_stride, dt), rk = heads_of(k, rows, Hkv, dh, k_stride, dt);
  const Rows rv = heads_of(v, v ? rows : 0, Hkv, dh, v_stride, dt);
  const Rows oq = heads_of(q_out, rows, Hq, dh, q_out_stride, dt);
  const Rows ok = heads_of(k_out, k_out ? rows : 0, Hkv, dh, k_out_stride, dt);
  const size_t pool = static_cast<size_t>(n_slots) * Hkv * dh * e;
  const Rows outs[] = {oq, ok, flat(k_pages, pool), flat(v_pages, pool)};
  const size_t vecb = static_cast<size_t>(dh) * sizeof(float);
  const Rows ins[] = {rq, rk, rv, flat(q_w, vecb), flat(k_w, vecb),
                      flat(inv_freq, static_cast<size_t>(rot) / 2 * sizeof(float)),
                      flat(positions, static_cast<size_t>(rows) * sizeof(int)),
                      flat(slots, static_cast<size_t>(rows) * sizeof(long long))};
  for (size_t i = 0; i < 4; ++i) {
    for (size_t j = 0; j < sizeof(ins) / sizeof(ins[0]); ++j)
      if (!(i == j && i < 2 && same(outs[i], ins[j])) && overlaps(outs[i], ins[j]))
        return RGLRU_ERR_INVALID_ARG;
    for (size_t j = i + 1; j < 4; ++j)
      if (overlaps(outs[i], outs[j])) return RGLRU_ERR_INVALID_ARG;
  }
  const rglru::RopeArgs a = {q,     k,        v,        q_w,      k_w,          inv_freq,
                             positions, slots, q_out,    k_out,    k_pages,      v_pages,
                             rows,  Hq,       Hkv,      dh,       rot,          q_stride,
                             k_stride, v_stride, q_out_stride, k_out_stride, n_slots, eps};
  (void)hipGetLastError();
  return hip_status(rglru::launch_qk_rope(a, dt == RGLRU_BF16 ? kBF16 : kF32,
                                          static_cast<hipStream_t>(stream)));
}

size_t rglru_qk_norm_rope_backward_workspace_size(int rows, int dh) {
  if (rows < 1 || dh < 1 || dh > rglru::kRopeMaxDh) return 0;
  return static_cast<size_t>(rglru::rope_bwd_groups(rows)) * 2 * dh * sizeof(float);
}

rglru_status rglru_qk_norm_rope_backward(const void *q, const void *k, const float *q_w,
                                         const float *k_w, const float *inv_freq,
                                         const int *positions, const void *dq_out,
                                         const void *dk_out, void *dq, void *dk, float *dq_w,
                                         float *dk_w, int rows, int Hq, int Hkv, int dh, int rot,
                                         long long q_stride, long long k_stride,
                                         long long dq_out_stride, long long dk_out_stride,
                                         long long dq_stride, long long dk_stride, float eps,
                                         rglru_dtype dt, void *workspace, size_t workspace_bytes,
                                         void *stream) {
  rglru_status st = check_rope(rows, Hq, Hkv, dh, rot, eps, dt, q_w, k_w, inv_freq);
  if (st != RGLRU_OK) return st;
  if (!q || !k || !positions || !dq_out || !dk_out || !dq || !dk) return RGLRU_ERR_INVALID_ARG;
  if (q_w && (!dq_w || !dk_w)) return RGLRU_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, Hq, dh) || !stride_ok(k_stride, Hkv, dh) ||
      !stride_ok(dq_out_stride, Hq, dh) || !stride_ok(dk_out_stride, Hkv, dh) ||
      !stride_ok(dq_stride, Hq, dh) || !stride_ok(dk_stride, Hkv, dh))
    return RGLRU_ERR_INVALID_ARG;
  const size_t e = elem_bytes(dt);
  const void *vec[] = {q, k, dq_out, dk_out, dq, dk};
  for (const void *p : vec)
    if (!aligned(p, e)) return RGLRU_ERR_INVALID_ARG;
  const void *vec4[] = {q_w, k_w, inv_freq, positions, dq_w, dk_w};
  for (const void *p : vec4)
    if (!aligned(p, 4)) return RGLRU_ERR_INVALID_ARG;
  const size_t need = q_w ? rglru_qk_norm_rope_backward_workspace_size(rows, dh) : 0;
  if (need && (!workspace || workspace_bytes < need)) return RGLRU_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return RGLRU_ERR_INVALID_ARG;
  const size_t vecb = static_cast<size_t>(dh) * sizeof(float);
  const Rows outs[] = {heads_of(dq, rows, Hq, dh, dq_stride, dt),
                       heads_of(dk, rows, Hkv, dh, dk_stride, dt), flat(q_w ? dq_w : nullptr, vecb),
                       flat(q_w ? dk_w : nullptr, vecb), flat(need ? workspace : nullptr, need)};
  const Rows ins[] = {heads_of(dq_out, rows, Hq, dh, dq_out_stride, dt),
                      heads_of(dk_out, rows, Hkv, dh, dk_out_stride, dt),
                      heads_of(q, rows, Hq, dh, q_stride, dt), heads_of(k, rows, Hkv, dh, k_stride, dt),
                      flat(q_w, vecb), flat(k_w, vecb),
                      flat(inv_freq, static_cast<size_t>(rot) / 2 * sizeof(float)),
                      flat(positions, static_cast<size_t>(rows) * sizeof(int))};
  for (size_t i = 0; i < 5; ++i) {
    for (size_t j = 0; j < sizeof(ins) / sizeof(ins[0]); ++j)
      if (!(i == j && i < 2 && same(outs[i], ins[j])) && overlaps(outs[i], ins[j]))
        return RGLRU_ERR_INVALID_ARG;
    for (size_t j = i + 1; j < 5; ++j)
      if (overlaps(outs[i], outs[j])) return RGLRU_ERR_INVALID_ARG;
  }
  const rglru::RopeBwdArgs a = {q,        k,        q_w,           k_w,           inv_freq,
                                positions, dq_out,  dk_out,        dq,            dk,
                                static_cast<float *>(workspace),   rows,          Hq,
                                Hkv,      dh,       rot,           q_stride,      k_stride,
                                dq_out_stride, dk_out_stride, dq_stride, dk_stride, eps};
  (void)hipGetLastError();
  return hip_status(rglru::launch_qk_rope_backward(a, dq_w, dk_w, dt == RGLRU_BF16 ? kBF16 : kF32,
                                                   static_cast<hipStream_t>(stream)));
}

rglru_status rglru_local_attention(const void *q, const void *k, const void *v, const int *lens,
                                   void *o, float *lse, int B, int T, int Hq, int Hkv, int dh,
                                   long long q_stride, long long k_stride, long long v_stride,
                                   int window, int sinks, float scale, rglru_dtype dt,
                                   void *stream) {
  rglru_status st =
      check_attn(B, T, Hq, Hkv, dh, q_stride, k_stride, v_stride, window, sinks, scale, dt);
  if (st != RGLRU_OK) return st;
  if (!q || !k || !v || !o) return RGLRU_ERR_INVALID_ARG;
  const void *vec16[] = {q, k, v, o};
  for (const void *p : vec16)
    if (!aligned(p, 16)) return RGLRU_ERR_INVALID_ARG;
  if (!aligned(lens, 4) || !aligned(lse, 4)) return RGLRU_ERR_INVALID_ARG;
  const size_t rows = static_cast<size_t>(B) * T;
  const Rows outs[] = {flat(o, rows * Hq * dh * 2), flat(lse, rows * Hq * sizeof(float))};
  const Rows ins[] = {heads_of(q, rows, Hq, dh, q_stride, dt), heads_of(k, rows, Hkv, dh, k_stride, dt),
                      heads_of(v, rows, Hkv, dh, v_stride, dt),
                      flat(lens, static_cast<size_t>(B) * sizeof(int))};
  for (const Rows &w : outs)
    for (const Rows &r : ins)
      if (overlaps(w, r)) return RGLRU_ERR_INVALID_ARG;
  if (overlaps(outs[0], outs[1])) return RGLRU_ERR_INVALID_ARG;
  if (scale == 0.0f) scale = 1.0f / std::sqrt(static_cast<float>(dh));
  const rglru::AttnArgs a = {q, k, v, o, lse, lens, B, T, Hq, Hkv, dh, q_stride, k_stride, v_stride,
                             window, sinks, scale, max_floor(scale * 1.4426950408889634f)};
  (void)hipGetLastError();
  return hip_status(rglru::launch_local_attention(a, static_cast<hipStream_t>(stream)));
}

size_t rglru_local_attention_backward_workspace_size(int B, int T, int Hq, int Hkv, int dh,
                                                     int window, int sinks) {
  if (check_attn(B, T, Hq, Hkv, dh, static_cast<long long>(Hq) * dh, static_cast<long long>(Hkv) * dh,
                 static_cast<long long>(Hkv) * dh, window, sinks, 0.0f, RGLRU_BF16) != RGLRU_OK ||
      !bwd_grid_ok(B, T, Hkv, dh))
    return 0;
  return attn_bwd_layout(rglru::attn_bwd_plan(B, T, Hq, Hkv, std::min(window, T), sinks), B, T, Hq, Hkv, dh).total;
}

rglru_status rglru_local_attention_backward(
    const void *q, const void *k, const void *v, const int *lens, const void *o, const float *lse,
    const void *d_o, void *dq, void *dk, void *dv, int B, int T, int Hq, int Hkv, int dh,
    long long q_stride, long long k_stride, long long v_stride, long long dq_stride,
    long long dk_stride, long long dv_stride, int window, int sinks, float scale, rglru_dtype dt,
    void *workspace, size_t workspace_bytes, void *stream) {
  rglru_status st =
      check_attn(B, T, Hq, Hkv, dh, q_stride, k_stride, v_stride, window, sinks, scale, dt);
  if (st != RGLRU_OK) return st;
  if (!bwd_grid_ok(B, T, Hkv, dh)) return RGLRU_ERR_UNSUPPORTED;
  if (!q || !k || !v || !o || !lse || !d_o || !dq || !dk || !dv) return RGLRU_ERR_INVALID_ARG;
  if (!stride_ok(dq_stride, Hq, dh) || !stride_ok(dk_stride, Hkv, dh) || !stride_ok(dv_stride, Hkv, dh))
    return RGLRU_ERR_INVALID_ARG;
  if (dq_stride % 8 || dk_stride % 8 || dv_stride % 8) return RGLRU_ERR_INVALID_ARG;
  const void *vec16[] = {q, k, v, o, d_o, dq, dk, dv};
  for (const void *p : vec16)
    if (!aligned(p, 16)) return RGLRU_ERR_INVALID_ARG;
  if (!aligned(lens, 4) || !aligned(lse, 4)) return RGLRU_ERR_INVALID_ARG;
  const size_t need = rglru_local_attention_backward_workspace_size(B, T, Hq, Hkv, dh, window, sinks);
  if (!workspace || workspace_bytes < need) return RGLRU_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return RGLRU_ERR_INVALID_ARG;
  const size_t rows = static_cast<size_t>(B) * T;
  const size_t obytes = rows * Hq * dh * 2;
  const Rows outs[] = {heads_of(dq, rows, Hq, dh, dq_stride, dt), heads_of(dk, rows, Hkv, dh, dk_stride, dt),
                       heads_of(dv, rows, Hkv, dh, dv_stride, dt), flat(workspace, need)};
  const Rows ins[] = {heads_of(q, rows, Hq, dh, q_stride, dt), heads_of(k, rows, Hkv, dh, k_stride, dt),
                      heads_of(v, rows, Hkv, dh, v_stride, dt), flat(o, obytes), flat(d_o, obytes),
                      flat(lse, rows * Hq * sizeof(float)),
                      flat(lens, static_cast<size_t>(B) * sizeof(int))};
  for (size_t i = 0; i < 4; ++i) {
    for (const Rows &r : ins)
      if (overlaps(outs[i], r)) return RGLRU_ERR_INVALID_ARG;
    for (size_t j = i + 1; j < 4; ++j)
      if (overlaps(outs[i], outs[j])) return RGLRU_ERR_INVALID_ARG;
  }
  if (scale == 0.0f) scale = 1.0f / std::sqrt(static_cast<float>(dh));
  window = std::min(window, T);
  sinks = std::min(sinks, T);
  const rglru::AttnBwdPlan p = rglru::attn_bwd_plan(B, T, Hq, Hkv, window, sinks);
  const AttnBwdLayout at = attn_bwd_layout(p, B, T, Hq, Hkv, dh);
  char *ws = static_cast<char *>(workspace);
  rglru::AttnBwdArgs a = {};
  a.q = q, a.k = k, a.v = v, a.o = o, a.do_ = d_o, a.lse = lse, a.lens = lens;
  a.dq = dq, a.dk = dk, a.dv = dv;
  a.lse2 = reinterpret_cast<float *>(ws);
  a.delta = reinterpret_cast<float *>(ws + at.delta);
  a.part = reinterpret_cast<float *>(ws + at.part);
  a.first = reinterpret_cast<long long *>(ws + at.first);
  a.span = reinterpret_cast<int2 *>(ws + at.span);
  a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.group = Hq / Hkv;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.dq_stride = dq_stride, a.dk_stride = dk_stride, a.dv_stride = dv_stride;
  a.window = window, a.sinks = sinks, a.scale = scale, a.c = scale * 1.4426950408889634f;
  a.groups = p.groups;
  (void)hipGetLastError();
  return hip_status(
      rglru::launch_local_attention_backward(a, dh, static_cast<hipStream_t>(stream)));
}

size_t rglru_paged_attention_workspace_size(int N, int Hq, int Hkv, int dh, int page_size,
                                            int max_pages, int window, int sinks, rglru_dtype dt) {
  if (check_paged(N, Hq, Hkv, dh, page_size, max_pages, window, sinks, dt) != RGLRU_OK) return 0;
  return paged_bytes(plan_of(N, Hq, Hkv, page_size, max_pages, window, sinks, dt), N, Hq, dh);
}

rglru_status rglru_paged_attention(const void *q, const void *k_pages, const void *v_pages,
                                   const int *block_table, const int *lens, void *o, int N, int Hq,
                                   int Hkv, int dh, long long q_stride, int num_pages,
                                   int page_size, int max_pages, int window, int sinks,
                                   float scale, rglru_dtype dt, void *workspace,
                                   size_t workspace_bytes, void *stream) {
  return paged_attention(q, k_pages, v_pages, nullptr, nullptr, block_table, lens, o, N, Hq, Hkv, dh, q_stride,
                         num_pages, page_size, max_pages, window, sinks, scale, dt, workspace, workspace_bytes, stream);
}

size_t rglru_paged_attention_e4m3_workspace_size(int N, int Hq, int Hkv, int dh, int page_size, int max_pages,
                                                 int window, int sinks) {
  return rglru_paged_attention_workspace_size(N, Hq, Hkv, dh, page_size, max_pages, window, sinks, RGLRU_BF16);
}

rglru_status rglru_paged_attention_e4m3(const void *q, const void *k_pages, const void *v_pages, const void *k_scales,
                                        const void *v_scales, const int *block_table, const int *lens, void *o, int N,
                                        int Hq, int Hkv, int dh, long long q_stride, int num_pages, int page_size,
                                        int max_pages, int window, int sinks, float scale, void *workspace,
                                        size_t workspace_bytes, void *stream) {
  if (!k_scales || !v_scales) return RGLRU_ERR_INVALID_ARG;
  return paged_attention(q, k_pages, v_pages, k_scales, v_scales, block_table, lens, o, N, Hq, Hkv, dh, q_stride,
                         num_pages, page_size, max_pages, window, sinks, scale, RGLRU_BF16, workspace,
                         workspace_bytes, stream);
}

size_t rglru_prefix_attention_workspace_size(int N, int Hq, int Hkv, int dh, int page_size, int prefix_pages,
                                             int max_pages, int window, int sinks) {
  if (check_prefix(N, Hq, Hkv, dh, page_size, prefix_pages, max_pages, window, sinks) != RGLRU_OK) return 0;
  return prefix_plans(N, Hq, Hkv, dh, page_size, prefix_pages, max_pages, window, sinks).bytes;
}

rglru_status rglru_prefix_attention(const void *q, const void *k_pages, const void *v_pages, const void *k_scales,
                                    const void *v_scales, const int *prefix_table, const int *prefix_len,
                                    const int *block_table, const int *lens, void *o, int N, int Hq, int Hkv, int dh,
                                    long long q_stride, int num_pages, int page_size, int prefix_pages, int max_pages,
                                    int window, int sinks, float scale, rglru_dtype dt, void *workspace,
                                    size_t workspace_bytes, void *stream) {
  if (dt != RGLRU_BF16) return RGLRU_ERR_UNSUPPORTED;
  const rglru_status st = check_prefix(N, Hq, Hkv, dh, page_size, prefix_pages, max_pages, window, sinks);
  if (st != RGLRU_OK) return st;
  if (!prefix_table || !prefix_len || (k_scales == nullptr) != (v_scales == nullptr)) return RGLRU_ERR_INVALID_ARG;
  if (!aligned(prefix_table, 4) || !aligned(prefix_len, 4)) return RGLRU_ERR_INVALID_ARG;
  const PrefixPlans plan = prefix_plans(N, Hq, Hkv, dh, page_size, prefix_pages, max_pages, window, sinks);
  const rglru_status sp = check_paged_tensors(q, k_pages, v_pages, k_scales, v_scales, block_table, lens, o, N, Hq, Hkv,
                                              dh, q_stride, num_pages, page_size, max_pages, scale, RGLRU_BF16,
                                              workspace, workspace_bytes, plan.bytes);
  if (sp != RGLRU_OK) return sp;
  const Rows outs[] = {flat(o, static_cast<size_t>(N) * Hq * dh * 2), flat(workspace, plan.bytes)};
  const Rows ins[] = {flat(prefix_table, static_cast<size_t>(prefix_pages) * sizeof(int)), flat(prefix_len, sizeof(int))};
  for (const Rows &w : outs)
    for (const Rows &r : ins)
      if (overlaps(w, r)) return RGLRU_ERR_INVALID_ARG;
  if (scale == 0.0f) scale = 1.0f / std::sqrt(static_cast<float>(dh));
  const float c = scale * 1.4426950408889634f;
  const long long cap = static_cast<long long>(prefix_pages) * page_size;
  float *const part = static_cast<float *>(workspace);
  float *const stat = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.part_bytes);
  const int parts = plan.shared.splits + plan.own.splits;
  const rglru::PagedArgs own = {q,         k_pages,   v_pages, block_table, lens,     o,        part,
                                stat,      N,         Hq,      Hkv,         dh,       q_stride, num_pages,
                                page_size, max_pages, window,  sinks,       c,        max_floor(c), k_scales,
                                v_scales,  prefix_len, cap,    parts,       plan.shared.splits};
  const rglru::PrefixArgs a = {q,    k_pages,  v_pages, k_scales,  v_scales,  prefix_table, prefix_len, lens, o,
                               part, stat,     N,       Hq,        Hkv,       q_stride,     cap,        num_pages,
                               page_size, parts, window, sinks,    c,         max_floor(c)};
  (void)hipGetLastError();
  return hip_status(rglru::launch_prefix_attention(a, own, plan.shared, plan.own, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
