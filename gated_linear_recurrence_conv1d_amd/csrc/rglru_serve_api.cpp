// rglru_serve_api.cpp -- the C ABI of the e4m3 cache's writing and reading and of linear attention (include/rglru.h):
// argument checks and kernel launches. No allocation, no global state; every call is asynchronous on its stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

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
using rglru::overlaps;
using rglru::Rows;
using rglru::stride_ok;

// Whether an output shares a byte with an input or another output.
template <size_t NO, size_t NI> bool clash(const Rows (&outs)[NO], const Rows (&ins)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (const Rows &r : ins)
      if (overlaps(outs[i], r)) return true;
    for (size_t j = i + 1; j < NO; ++j)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}

bool rows_16b(const void *p, long long stride, int heads, int dh, size_t e) {
  return aligned(p, 16) && stride_ok(stride, heads, dh) && stride * e % 16 == 0;
}

bool dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

rglru_status check_linear(int rows, int Hk, int H, int dk, int dv, long long q_stride, long long k_stride,
                          long long v_stride, float scale, rglru_dtype dt) {
  if (rows < 1 || Hk < 1 || H < 1 || dk < 1 || dv < 1 || H % Hk) return RGLRU_ERR_INVALID_ARG;
  if (!(scale == scale) || scale < 0.0f || std::isinf(scale)) return RGLRU_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, Hk, dk) || !stride_ok(k_stride, Hk, dk) || !stride_ok(v_stride, H, dv))
    return RGLRU_ERR_INVALID_ARG;
  if (q_stride % 8 || k_stride % 8 || v_stride % 8) return RGLRU_ERR_INVALID_ARG;
  if (dt != RGLRU_BF16 || !dim_ok(dk) || !dim_ok(dv) || H > 65535) return RGLRU_ERR_UNSUPPORTED;
  if (q_stride > kMaxStride || k_stride > kMaxStride || v_stride > kMaxStride) return RGLRU_ERR_UNSUPPORTED;
  // workgroups of 32 values of a state, or of 256 times 4 values of all states
  if (static_cast<long long>(rows) * H * 64 >= rglru::kMaxBlocks) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

rglru_status check_prompt(int B, int T, int Hk, int H, int dk, int dv, long long q_stride, long long k_stride,
                          long long v_stride, float scale, rglru_dtype dt) {
  if (T < 1) return RGLRU_ERR_INVALID_ARG;
  const rglru_status st = check_linear(B, Hk, H, dk, dv, q_stride, k_stride, v_stride, scale, dt);
  if (st != RGLRU_OK) return st;
  return T >= kMaxTokens ? RGLRU_ERR_UNSUPPORTED : RGLRU_OK;
}

// The segments' states, then their decays.
size_t seg_bytes(const rglru::LinearPlan &p, int B, int H, int dk, int dv) {
  return rglru::align_up(static_cast<size_t>(B) * H * (p.states + 1) * dk * dv * sizeof(float));
}
size_t linear_bytes(const rglru::LinearPlan &p, int B, int H, int dk, int dv) {
  if (!p.states) return 0;
  return seg_bytes(p, B, H, dk, dv) + rglru::align_up(static_cast<size_t>(B) * H * p.states * sizeof(float));
}

}  // namespace

extern "C" {

rglru_status rglru_cache_quantize(const void *k, const void *v, const long long *slots, void *k_pages, void *v_pages,
                                  void *k_scales, void *v_scales, int rows, int Hkv, int dh, long long k_stride,
                                  long long v_stride, long long n_slots, rglru_dtype dt, void *stream) {
  const rglru_status st = check_heads(rows, Hkv, Hkv, dh, dt);
  if (st != RGLRU_OK) return st;
  if (n_slots < 1) return RGLRU_ERR_INVALID_ARG;
  if (!dim_ok(dh) || n_slots >= kMaxTokens) return RGLRU_ERR_UNSUPPORTED;
  if (static_cast<long long>(rows) * Hkv * (dh / 8) / 256 >= rglru::kMaxBlocks) return RGLRU_ERR_UNSUPPORTED;
  if (!k || !v || !slots || !k_pages || !v_pages || !k_scales || !v_scales) return RGLRU_ERR_INVALID_ARG;
  const size_t e = elem_bytes(dt);
  if (!rows_16b(k, k_stride, Hkv, dh, e) || !rows_16b(v, v_stride, Hkv, dh, e)) return RGLRU_ERR_INVALID_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(slots, 8)) return RGLRU_ERR_INVALID_ARG;
  const size_t heads = static_cast<size_t>(n_slots) * Hkv;
  const Rows outs[] = {flat(k_pages, heads * dh), flat(v_pages, heads * dh), flat(k_scales, heads), flat(v_scales, heads)};
  const Rows ins[] = {heads_of(k, rows, Hkv, dh, k_stride, dt), heads_of(v, rows, Hkv, dh, v_stride, dt),
                      flat(slots, static_cast<size_t>(rows) * sizeof(long long))};
  if (clash(outs, ins)) return RGLRU_ERR_INVALID_ARG;
  const rglru::CacheWriteArgs a = {k, v, slots, k_pages, v_pages, k_scales, v_scales, rows, Hkv, k_stride, v_stride,
                                   n_slots};
  (void)hipGetLastError();
  return hip_status(
      rglru::launch_cache_quantize(a, dh, dt == RGLRU_BF16 ? kBF16 : kF32, static_cast<hipStream_t>(stream)));
}

rglru_status rglru_cache_dequantize(const void *k_pages, const void *v_pages, const void *k_scales,
                                    const void *v_scales, const int *block_table, const int *lens, const int *starts,
                                    void *k_out, void *v_out, int B, int T, int Hkv, int dh, long long k_stride,
                                    long long v_stride, int num_pages, int page_size, int max_pages, int zero_rest,
                                    rglru_dtype dt, void *stream) {
  const rglru_status st = check_heads(B, Hkv, Hkv, dh, dt);
  if (st != RGLRU_OK) return st;
  if (T < 1 || num_pages < 1 || page_size < 1 || max_pages < 1) return RGLRU_ERR_INVALID_ARG;
  if (!dim_ok(dh)) return RGLRU_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * page_size >= kMaxTokens ||
      static_cast<long long>(max_pages) * page_size >= kMaxTokens || T >= kMaxTokens)
    return RGLRU_ERR_UNSUPPORTED;
  const long long blocks = rglru::cache_read_blocks(T, Hkv, dh);
  if (blocks >= rglru::kMaxBlocks || blocks * B >= rglru::kMaxBlocks) return RGLRU_ERR_UNSUPPORTED;
  if (!k_pages || !v_pages || !k_scales || !v_scales || !block_table || !lens || !k_out || !v_out)
    return RGLRU_ERR_INVALID_ARG;
  const size_t e = elem_bytes(dt);
  if (!rows_16b(k_out, k_stride, Hkv, dh, e) || !rows_16b(v_out, v_stride, Hkv, dh, e)) return RGLRU_ERR_INVALID_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(block_table, 4) || !aligned(lens, 4) ||
      !aligned(starts, 4))
    return RGLRU_ERR_INVALID_ARG;
  const size_t heads = static_cast<size_t>(num_pages) * page_size * Hkv, rows = static_cast<size_t>(B) * T;
  const Rows outs[] = {heads_of(k_out, rows, Hkv, dh, k_stride, dt), heads_of(v_out, rows, Hkv, dh, v_stride, dt)};
  const Rows ins[] = {flat(k_pages, heads * dh), flat(v_pages, heads * dh), flat(k_scales, heads), flat(v_scales, heads),
                      flat(block_table, static_cast<size_t>(B) * max_pages * sizeof(int)),
                      flat(lens, static_cast<size_t>(B) * sizeof(int)),
                      flat(starts, static_cast<size_t>(B) * sizeof(int))};
  if (clash(outs, ins)) return RGLRU_ERR_INVALID_ARG;
  const rglru::CacheReadArgs a = {k_pages, v_pages, k_scales, v_scales, block_table, lens,      starts,    k_out,    v_out,
                                  B,       T,       Hkv,      k_stride, v_stride,    num_pages, page_size, max_pages,
                                  zero_rest != 0};
  (void)hipGetLastError();
  return hip_status(
      rglru::launch_cache_dequantize(a, dh, dt == RGLRU_BF16 ? kBF16 : kF32, static_cast<hipStream_t>(stream)));
}

size_t rglru_linear_attention_workspace_size(int B, int T, int Hk, int H, int dk, int dv) {
  if (check_prompt(B, T, Hk, H, dk, dv, static_cast<long long>(Hk) * dk, static_cast<long long>(Hk) * dk,
                   static_cast<long long>(H) * dv, 0.0f, RGLRU_BF16) != RGLRU_OK)
    return 0;
  return linear_bytes(rglru::linear_plan(B, T, H, dk, dv), B, H, dk, dv);
}

rglru_status rglru_linear_attention(const void *q, const void *k, const void *v, const float *log_decay,
                                    const int *lens, const float *s0, void *o, float *s_out, int B, int T, int Hk,
                                    int H, int dk, int dv, long long q_stride, long long k_stride, long long v_stride,
                                    int gated, float scale, rglru_dtype dt, void *workspace, size_t workspace_bytes,
                                    void *stream) {
  const rglru_status st = check_prompt(B, T, Hk, H, dk, dv, q_stride, k_stride, v_stride, scale, dt);
  if (st != RGLRU_OK) return st;
  if (!q || !k || !v || !log_decay || !o) return RGLRU_ERR_INVALID_ARG;
  const void *vec16[] = {q, k, v, o, s0, s_out};
  for (const void *p : vec16)
    if (!aligned(p, 16)) return RGLRU_ERR_INVALID_ARG;
  if (!aligned(log_decay, 4) || !aligned(lens, 4)) return RGLRU_ERR_INVALID_ARG;
  const rglru::LinearPlan plan = rglru::linear_plan(B, T, H, dk, dv);
  const size_t need = linear_bytes(plan, B, H, dk, dv);
  if (need && (!workspace || workspace_bytes < need)) return RGLRU_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return RGLRU_ERR_INVALID_ARG;
  const size_t rows = static_cast<size_t>(B) * T, state = static_cast<size_t>(B) * H * dk * dv * sizeof(float);
  const Rows s_in = flat(s0, state), outs[] = {flat(o, rows * H * dv * 2), flat(s_out, state),
                                               flat(need ? workspace : nullptr, need)};
  const Rows ins[] = {heads_of(q, rows, Hk, dk, q_stride, dt), heads_of(k, rows, Hk, dk, k_stride, dt),
                      heads_of(v, rows, H, dv, v_stride, dt),
                      flat(log_decay, (gated ? rows : 1) * H * sizeof(float)),
                      flat(lens, static_cast<size_t>(B) * sizeof(int)),
                      s_out == s0 ? flat(nullptr, 0) : s_in};
  if (clash(outs, ins) || overlaps(outs[0], s_in) || overlaps(outs[2], s_in)) return RGLRU_ERR_INVALID_ARG;
  if (scale == 0.0f) scale = 1.0f / std::sqrt(static_cast<float>(dk));
  char *const ws = static_cast<char *>(workspace);
  rglru::LinearArgs a = {};
  a.q = q, a.k = k, a.v = v, a.log_decay = log_decay, a.lens = lens, a.s0 = s0, a.o = o, a.s_out = s_out;
  if (need) {
    a.seg = reinterpret_cast<float *>(ws);
    a.sums = reinterpret_cast<float *>(ws + seg_bytes(plan, B, H, dk, dv));
  }
  a.B = B, a.T = T, a.Hk = Hk, a.H = H, a.dk = dk, a.dv = dv;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.scale = scale, a.gated = gated != 0, a.segs = plan.segs, a.sub = plan.sub, a.states = plan.states;
  a.seg_len = plan.seg_len;
  (void)hipGetLastError();
  return hip_status(rglru::launch_linear_attention(a, static_cast<hipStream_t>(stream)));
}

rglru_status rglru_linear_attention_step(const void *q, const void *k, const void *v, const float *log_decay,
                                         const float *s_in, float *s_out, void *o, int N, int Hk, int H, int dk, int dv,
                                         long long q_stride, long long k_stride, long long v_stride, int gated,
                                         float scale, rglru_dtype dt, void *stream) {
  const rglru_status st = check_linear(N, Hk, H, dk, dv, q_stride, k_stride, v_stride, scale, dt);
  if (st != RGLRU_OK) return st;
  if (!q || !k || !v || !log_decay || !s_in || !s_out || !o) return RGLRU_ERR_INVALID_ARG;
  const void *vec16[] = {q, k, v, o, s_in, s_out};
  for (const void *p : vec16)
    if (!aligned(p, 16)) return RGLRU_ERR_INVALID_ARG;
  if (!aligned(log_decay, 4)) return RGLRU_ERR_INVALID_ARG;
  const size_t rows = N, state = static_cast<size_t>(N) * H * dk * dv * sizeof(float);
  const Rows in = flat(s_in, state), outs[] = {flat(o, rows * H * dv * 2), flat(s_out, state)};
  const Rows ins[] = {heads_of(q, rows, Hk, dk, q_stride, dt), heads_of(k, rows, Hk, dk, k_stride, dt),
                      heads_of(v, rows, H, dv, v_stride, dt), flat(log_decay, (gated ? rows : 1) * H * sizeof(float)),
                      s_out == s_in ? flat(nullptr, 0) : in};
  if (clash(outs, ins) || overlaps(outs[0], in)) return RGLRU_ERR_INVALID_ARG;
  if (scale == 0.0f) scale = 1.0f / std::sqrt(static_cast<float>(dk));
  const rglru::LinearStepArgs a = {q, k, v, log_decay, s_in, s_out, o, N, Hk, H, dk, dv, q_stride, k_stride, v_stride,
                                   scale, gated != 0};
  (void)hipGetLastError();
  return hip_status(rglru::launch_linear_step(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
