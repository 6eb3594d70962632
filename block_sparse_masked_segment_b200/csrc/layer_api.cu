// layer_api.cu - the extern "C" entry points of the operators around the
// attention (rotary positions, per-head norm with rotation, matrix product with
// epilogue): host-side argument checks and dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "host_status.h"
#include "layer.cuh"
#include "opr_internal.cuh"

namespace opr {
namespace {

constexpr int64_t kMaxRows = int64_t{1} << 31;
constexpr int32_t kMaxHeads = 65536;

// A strided block of rows in memory.
struct Rows {
  const void* p;
  int64_t rows, stride, width;  // elements
  int32_t dtype;
  int64_t step() const { return stride * dtype_bytes(dtype); }
  int64_t bytes() const { return rows <= 0 ? 0 : (rows - 1) * step() + width * dtype_bytes(dtype); }
  bool same(const Rows& o) const { return p == o.p && dtype == o.dtype && stride == o.stride; }
};

// An array of n 32-bit words as one row.
Rows words(const void* p, int64_t n) { return {p, 1, n, n, OPR_DTYPE_FP32}; }

// May the two share memory?  Blocks of rows with one stride, side by side in
// wider rows, do not although their ranges do, nor does a single row between those
// of a block.
bool overlap(const Rows& a, const Rows& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes() == 0 || b.bytes() == 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  if (pa + static_cast<uint64_t>(a.bytes()) <= pb || pb + static_cast<uint64_t>(b.bytes()) <= pa) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.rows != 1 && b.rows != 1 && a.step() != b.step()) return true;
  const int64_t step = a.rows == 1 ? b.step() : a.step();
  const int64_t wa = a.width * dtype_bytes(a.dtype), wb = b.width * dtype_bytes(b.dtype);
  const int64_t diff = pb >= pa ? static_cast<int64_t>((pb - pa) % static_cast<uint64_t>(step))
                                : step - 1 - static_cast<int64_t>((pa - pb - 1) % static_cast<uint64_t>(step));
  return !(diff >= wa && diff + wb <= step);
}

bool element_aligned(const void* p, int32_t dtype) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(dtype_bytes(dtype)) == 0;
}

// Arrays of 32 and of 64 bits, null allowed.
bool words_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool doubles_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// What the three calls on heads check alike.
bool head_arrays_ok(const int32_t* pos_id, const double* freq, const int32_t* row_map, const int32_t* dev_status) {
  return words_aligned(pos_id) && doubles_aligned(freq) && words_aligned(row_map) && words_aligned(dev_status);
}
bool head_args_ok(int64_t total, int32_t head_dim, int32_t rot_dim, float scale) {
  return total >= 0 && total < kMaxRows && head_dim >= 2 && head_dim <= 256 && rot_dim >= 2 && rot_dim % 2 == 0 &&
         rot_dim <= head_dim && std::isfinite(scale);
}

HeadArgs head_args(const int32_t* pos_id, const double* freq, int32_t rot_dim, int32_t interleaved, float scale,
                   const int32_t* row_map, int64_t total, int32_t head_dim, int32_t* dev_status) {
  HeadArgs a{};
  a.pos = pos_id;
  a.freq = freq;
  a.row_map = row_map;
  a.total = total;
  a.d = head_dim;
  a.pairs = rot_dim / 2;
  a.interleaved = interleaved != 0;
  a.scale = scale;
  a.dev_status = dev_status;
  return a;
}

// Does any output share memory with another output, or with an input other than
// the one it may replace (the same rows, and no row map)?
struct OutRows {
  Rows rows;
  const Rows* replaces[2];
};
template <int NI, int NO>
bool outputs_clash(const Rows (&in)[NI], const OutRows (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = i + 1; j < NO; ++j)
      if (overlap(out[i].rows, out[j].rows)) return true;
    for (int j = 0; j < NI; ++j) {
      if (!overlap(out[i].rows, in[j])) continue;
      const bool takes = out[i].replaces[0] == &in[j] || out[i].replaces[1] == &in[j];
      if (!(takes && out[i].rows.same(in[j]))) return true;
    }
  }
  return false;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// An operand of the matrix products is used where it lies when every row starts
// on a 16-byte boundary, else from a copy with padded rows.
bool tma_ready(const void* p, int64_t ld) { return aligned16(p) && ld % 8 == 0; }
int64_t padded(int64_t cols) { return (cols + 7) / 8 * 8; }
size_t copy_bytes(int64_t rows, int64_t cols) {
  return align_up(static_cast<size_t>(rows) * static_cast<size_t>(padded(cols)) * 2, 256);
}

// Points an operand at a copy with padded rows, and says what to copy.
PackJob pack(Operand& o, int64_t rows, int32_t cols, void* to) {
  const PackJob job{o.p, o.row, to, padded(cols), rows, cols};
  o = Operand{to, padded(cols), 1};
  return job;
}

// Coordinates of whole tiles past the ends stay within int32.
constexpr int64_t kMaxExtent = kMaxRows - 512;
bool linear_sizes_ok(int64_t m, int32_t n, int32_t k) {
  return m >= 0 && m <= kMaxExtent && n > 0 && n <= kMaxExtent && k > 0 && k <= kMaxExtent;
}
bool known_act(int32_t a) { return a >= OPR_ACT_NONE && a <= OPR_ACT_GELU_TANH; }

}  // namespace
}  // namespace opr

using namespace opr;

extern "C" {

opr_status opr_rotary_frequencies(int32_t rot_dim, double base, int32_t rule, double factor, double original_length,
                                  double low_turns, double high_turns, double* freq, double* scale) {
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 256 || !freq || !scale) return OPR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base)) return OPR_INVALID_ARG;
  if (rule < OPR_ROTARY_PLAIN || rule > OPR_ROTARY_WAVELENGTH) return OPR_UNSUPPORTED;
  if (rule != OPR_ROTARY_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return OPR_INVALID_ARG;
  if (rule == OPR_ROTARY_NTK && rot_dim == 2) return OPR_INVALID_ARG;  // one pair: its frequency is 1 at any base
  const bool ramped = rule == OPR_ROTARY_YARN || rule == OPR_ROTARY_WAVELENGTH;
  if (ramped && (!(original_length > 0.0) || !std::isfinite(original_length) || !(low_turns > 0.0) ||
                 !(high_turns > low_turns) || !std::isfinite(high_turns)))
    return OPR_INVALID_ARG;
  const double two_pi = 6.283185307179586;
  const int pairs = rot_dim / 2;
  if (rule == OPR_ROTARY_NTK) base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  *scale = rule == OPR_ROTARY_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  double lo = 0.0, hi = 0.0;
  if (rule == OPR_ROTARY_YARN) {  // pair indices that make high_turns and low_turns over the original length
    const double per = rot_dim / (2.0 * std::log(base));
    lo = std::fmax(std::floor(per * std::log(original_length / (two_pi * high_turns))), 0.0);
    hi = std::fmin(std::ceil(per * std::log(original_length / (two_pi * low_turns))), rot_dim - 1.0);
  }
  for (int j = 0; j < pairs; ++j) {
    double f = std::pow(base, -2.0 * j / rot_dim);
    if (rule == OPR_ROTARY_LINEAR) f /= factor;
    if (ramped) {
      // share of the original frequency that is kept
      double keep;
      if (rule == OPR_ROTARY_YARN)
        keep = 1.0 - std::fmin(std::fmax((j - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
      else
        keep = std::fmin(std::fmax((original_length * f / two_pi - low_turns) / (high_turns - low_turns), 0.0), 1.0);
      f = f * keep + f / factor * (1.0 - keep);
    }
    freq[j] = f;
  }
  return OPR_OK;
}

opr_status opr_rotary(const void* x, int32_t x_dtype, int64_t x_stride, void* y, int32_t y_dtype, int64_t y_stride,
                      const int32_t* pos_id, const double* freq, int32_t rot_dim, int32_t interleaved, float scale,
                      int32_t inverse, const int32_t* row_map, int64_t total_tokens, int32_t n_heads,
                      int32_t head_dim, int32_t* dev_status, void* stream) {
  CallRange range("opr_rotary");
  if (!head_args_ok(total_tokens, head_dim, rot_dim, scale) || n_heads < 0 || n_heads > kMaxHeads) return OPR_INVALID_ARG;
  if (!known_dtype(x_dtype) || !known_dtype(y_dtype)) return OPR_UNSUPPORTED;
  const int64_t width = static_cast<int64_t>(n_heads) * head_dim;
  if (x_stride < width || y_stride < width) return OPR_INVALID_ARG;
  if (total_tokens == 0 || n_heads == 0) return OPR_OK;
  if (!x || !y || !pos_id || !freq || !element_aligned(x, x_dtype) || !element_aligned(y, y_dtype) ||
      !head_arrays_ok(pos_id, freq, row_map, dev_status))
    return OPR_INVALID_ARG;
  const Rows in[4] = {{x, total_tokens, x_stride, width, x_dtype},
                      words(pos_id, total_tokens),
                      words(freq, rot_dim),  // rot_dim / 2 of 64 bits
                      words(row_map, total_tokens)};
  const OutRows out[1] = {{{y, total_tokens, y_stride, width, y_dtype}, {row_map ? nullptr : &in[0], nullptr}}};
  if (outputs_clash(in, out)) return OPR_INVALID_ARG;
  const opr_status st = device_check();
  if (st != OPR_OK) return st;
  HeadArgs a = head_args(pos_id, freq, rot_dim, interleaved, scale, row_map, total_tokens, head_dim, dev_status);
  a.inverse = inverse != 0;
  a.n_sets = 1;
  a.set[0].x = x;
  a.set[0].x_stride = x_stride;
  a.set[0].y = y;
  a.set[0].y_stride = y_stride;
  a.set[0].heads = n_heads;
  a.set[0].mode = kHeadRotate;
  return status_of(launch_heads(a, x_dtype, y_dtype, static_cast<cudaStream_t>(stream)));
}

opr_status opr_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, int32_t x_dtype, const void* q_weight, const void* k_weight,
                            int32_t w_dtype, float eps, const int32_t* pos_id, const double* freq, int32_t rot_dim,
                            int32_t interleaved, float scale, const int32_t* row_map, int64_t total_tokens, int32_t hq,
                            int32_t hkv, int32_t head_dim, void* q_out, void* k_out, void* v_out, int32_t y_dtype,
                            int32_t* dev_status, void* stream) {
  CallRange range("opr_qk_norm_rope");
  if (!head_args_ok(total_tokens, head_dim, rot_dim, scale) || hq <= 0 || hkv <= 0 || hq > kMaxHeads || hkv > kMaxHeads)
    return OPR_INVALID_ARG;
  if (!known_dtype(x_dtype) || !known_dtype(y_dtype) || !known_dtype(w_dtype)) return OPR_UNSUPPORTED;
  if (!(eps > 0.f) || !std::isfinite(eps)) return OPR_INVALID_ARG;
  const int64_t wq = static_cast<int64_t>(hq) * head_dim, wkv = static_cast<int64_t>(hkv) * head_dim;
  if (q_stride < wq || k_stride < wkv || (v && v_stride < wkv))
    return OPR_INVALID_ARG;
  if ((v == nullptr) != (v_out == nullptr)) return OPR_INVALID_ARG;
  if (total_tokens == 0) return OPR_OK;
  if (!q || !k || !q_weight || !k_weight || !pos_id || !freq || !q_out || !k_out) return OPR_INVALID_ARG;
  for (const void* p : {q, k, v})
    if (!element_aligned(p, x_dtype)) return OPR_INVALID_ARG;
  for (const void* p : {q_out, k_out, v_out})
    if (!element_aligned(p, y_dtype)) return OPR_INVALID_ARG;
  if (!element_aligned(q_weight, w_dtype) || !element_aligned(k_weight, w_dtype) ||
      !head_arrays_ok(pos_id, freq, row_map, dev_status))
    return OPR_INVALID_ARG;
  const Rows in[8] = {{q, total_tokens, q_stride, wq, x_dtype},
                      {k, total_tokens, k_stride, wkv, x_dtype},
                      {v, total_tokens, v_stride, wkv, x_dtype},
                      {q_weight, 1, head_dim, head_dim, w_dtype},
                      {k_weight, 1, head_dim, head_dim, w_dtype},
                      words(pos_id, total_tokens),
                      words(freq, rot_dim),
                      words(row_map, total_tokens)};
  const bool in_place = row_map == nullptr;
  const OutRows out[3] = {{{q_out, total_tokens, wq, wq, y_dtype}, {in_place ? &in[0] : nullptr, nullptr}},
                          {{k_out, total_tokens, wkv, wkv, y_dtype}, {in_place ? &in[1] : nullptr, nullptr}},
                          {{v_out, total_tokens, wkv, wkv, y_dtype}, {in_place ? &in[2] : nullptr, nullptr}}};
  if (outputs_clash(in, out)) return OPR_INVALID_ARG;
  const opr_status st = device_check();
  if (st != OPR_OK) return st;
  HeadArgs a = head_args(pos_id, freq, rot_dim, interleaved, scale, row_map, total_tokens, head_dim, dev_status);
  a.eps = eps;
  a.w_dtype = w_dtype;
  a.n_sets = v != nullptr ? 3 : 2;
  const void* xs[3] = {q, k, v};
  const int64_t strides[3] = {q_stride, k_stride, v_stride};
  void* ys[3] = {q_out, k_out, v_out};
  const void* ws[3] = {q_weight, k_weight, nullptr};
  for (int i = 0; i < a.n_sets; ++i) {
    a.set[i].x = xs[i];
    a.set[i].x_stride = strides[i];
    a.set[i].y = ys[i];
    a.set[i].heads = i == 0 ? hq : hkv;
    a.set[i].y_stride = i == 0 ? wq : wkv;
    a.set[i].w = ws[i];
    a.set[i].mode = i == 2 ? kHeadCopy : kHeadNormRotate;
  }
  return status_of(launch_heads(a, x_dtype, y_dtype, static_cast<cudaStream_t>(stream)));
}

size_t opr_qk_norm_rope_bwd_workspace_bytes(int64_t total_tokens, int32_t hq, int32_t hkv, int32_t head_dim) {
  if (total_tokens < 0 || total_tokens >= kMaxRows || hq <= 0 || hkv <= 0 || head_dim < 2 || head_dim > 256) return 0;
  const size_t blocks = static_cast<size_t>(head_grad_blocks(total_tokens, hq > hkv ? hq : hkv));
  return align_up(2 * (blocks > 0 ? blocks : 1) * static_cast<size_t>(head_dim) * sizeof(float), 256);
}

opr_status opr_qk_norm_rope_bwd(const void* dq, const void* dk, const void* dv, int32_t dy_dtype, const void* q,
                                int64_t q_stride, const void* k, int64_t k_stride, int32_t x_dtype,
                                const void* q_weight, const void* k_weight, int32_t w_dtype, float eps,
                                const int32_t* pos_id, const double* freq, int32_t rot_dim, int32_t interleaved,
                                float scale, const int32_t* row_map, int64_t total_tokens, int32_t hq, int32_t hkv,
                                int32_t head_dim, void* dq_out, int64_t dq_stride, void* dk_out, int64_t dk_stride,
                                void* dv_out, int64_t dv_stride, int32_t dx_dtype, float* dq_weight, float* dk_weight,
                                void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  CallRange range("opr_qk_norm_rope_bwd");
  if (!head_args_ok(total_tokens, head_dim, rot_dim, scale) || hq <= 0 || hkv <= 0 || hq > kMaxHeads || hkv > kMaxHeads)
    return OPR_INVALID_ARG;
  if (!known_dtype(x_dtype) || !known_dtype(dy_dtype) || !known_dtype(dx_dtype) || !known_dtype(w_dtype))
    return OPR_UNSUPPORTED;
  if (!(eps > 0.f) || !std::isfinite(eps)) return OPR_INVALID_ARG;
  const int64_t wq = static_cast<int64_t>(hq) * head_dim, wkv = static_cast<int64_t>(hkv) * head_dim;
  if (q_stride < wq || k_stride < wkv || dq_stride < wq || dk_stride < wkv ||
      (dv && dv_stride < wkv))
    return OPR_INVALID_ARG;
  if ((dv == nullptr) != (dv_out == nullptr)) return OPR_INVALID_ARG;
  if (!q_weight || !k_weight || !dq_weight || !dk_weight || !workspace) return OPR_INVALID_ARG;
  if (workspace_bytes < opr_qk_norm_rope_bwd_workspace_bytes(total_tokens, hq, hkv, head_dim))
    return OPR_WORKSPACE_TOO_SMALL;
  if (total_tokens > 0 && (!dq || !dk || !q || !k || !pos_id || !freq || !dq_out || !dk_out)) return OPR_INVALID_ARG;
  if (!aligned16(workspace) || !element_aligned(dq_weight, OPR_DTYPE_FP32) ||
      !element_aligned(dk_weight, OPR_DTYPE_FP32) || !element_aligned(q_weight, w_dtype) ||
      !element_aligned(k_weight, w_dtype) || !head_arrays_ok(pos_id, freq, row_map, dev_status))
    return OPR_INVALID_ARG;
  for (const void* p : {dq, dk, dv})
    if (!element_aligned(p, dy_dtype)) return OPR_INVALID_ARG;
  for (const void* p : {q, k})
    if (!element_aligned(p, x_dtype)) return OPR_INVALID_ARG;
  for (const void* p : {dq_out, dk_out, dv_out})
    if (!element_aligned(p, dx_dtype)) return OPR_INVALID_ARG;
  const int64_t n = total_tokens;
  const Rows in[10] = {{dq, n, wq, wq, dy_dtype},    {dk, n, wkv, wkv, dy_dtype},
                      {dv, n, wkv, wkv, dy_dtype},   {q, n, q_stride, wq, x_dtype},
                      {k, n, k_stride, wkv, x_dtype}, {q_weight, 1, head_dim, head_dim, w_dtype},
                      {k_weight, 1, head_dim, head_dim, w_dtype},
                      words(pos_id, n),              words(freq, rot_dim),
                      words(row_map, n)};
  const Rows* own_dy[3] = {&in[0], &in[1], &in[2]};
  if (row_map != nullptr) own_dy[0] = own_dy[1] = own_dy[2] = nullptr;
  const int64_t ws_words = static_cast<int64_t>(workspace_bytes / sizeof(float));
  const OutRows out[6] = {{{dq_out, n, dq_stride, wq, dx_dtype}, {own_dy[0], &in[3]}},
                          {{dk_out, n, dk_stride, wkv, dx_dtype}, {own_dy[1], &in[4]}},
                          {{dv_out, n, dv_stride, wkv, dx_dtype}, {own_dy[2], nullptr}},
                          {{dq_weight, 1, head_dim, head_dim, OPR_DTYPE_FP32}, {nullptr, nullptr}},
                          {{dk_weight, 1, head_dim, head_dim, OPR_DTYPE_FP32}, {nullptr, nullptr}},
                          {{workspace, 1, ws_words, ws_words, OPR_DTYPE_FP32}, {nullptr, nullptr}}};
  if (outputs_clash(in, out)) return OPR_INVALID_ARG;
  const opr_status st = device_check();
  if (st != OPR_OK) return st;
  HeadArgs a = head_args(pos_id, freq, rot_dim, interleaved, scale, row_map, total_tokens, head_dim, dev_status);
  a.eps = eps;
  a.w_dtype = w_dtype;
  a.n_sets = dv != nullptr ? 3 : 2;
  const void* dys[3] = {dq, dk, dv};
  const void* xs[3] = {q, k, nullptr};
  const int64_t x_strides[3] = {q_stride, k_stride, 0};
  void* dxs[3] = {dq_out, dk_out, dv_out};
  const int64_t dx_strides[3] = {dq_stride, dk_stride, dv_stride};
  const void* ws[3] = {q_weight, k_weight, nullptr};
  float* grads[3] = {dq_weight, dk_weight, nullptr};
  const int64_t blocks = head_grad_blocks(total_tokens, hq > hkv ? hq : hkv);
  for (int i = 0; i < a.n_sets; ++i) {
    HeadSet& s = a.set[i];
    s.x = xs[i];
    s.x_stride = x_strides[i];
    s.dy = dys[i];
    s.dy_stride = i == 0 ? wq : wkv;
    s.y = dxs[i];
    s.y_stride = dx_strides[i];
    s.w = ws[i];
    s.w_grad = grads[i];
    s.partial = i < 2 ? static_cast<float*>(workspace) + i * blocks * head_dim : nullptr;
    s.heads = i == 0 ? hq : hkv;
    s.mode = i == 2 ? kHeadCopy : kHeadNormRotate;
  }
  return status_of(launch_head_grads(a, x_dtype, dy_dtype, dx_dtype, static_cast<cudaStream_t>(stream)));
}

size_t opr_linear_workspace_bytes(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t m, int32_t n,
                                  int32_t k) {
  if (!linear_sizes_ok(m, n, k) || ldx < k || ldw < k) return 0;
  return (tma_ready(x, ldx) ? 0 : copy_bytes(m, k)) + (tma_ready(w, ldw) ? 0 : copy_bytes(n, k));
}

opr_status opr_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, int32_t dtype, const void* bias,
                      int32_t bias_dtype, int32_t activation, const void* residual, int64_t ld_residual,
                      int32_t residual_dtype, void* y, int64_t ldy, int32_t y_dtype, void* z, int64_t ldz, int64_t m,
                      int32_t n, int32_t k, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                      void* stream) {
  CallRange range("opr_linear");
  if (!linear_sizes_ok(m, n, k) || ldx < k || ldw < k || ldy < n || (residual && ld_residual < n) || (z && ldz < n))
    return OPR_INVALID_ARG;
  if (!known_act(activation)) return OPR_UNSUPPORTED;
  if (dtype != OPR_DTYPE_BF16 && dtype != OPR_DTYPE_FP16) return OPR_UNSUPPORTED;
  if (!known_dtype(y_dtype) || (bias && !known_dtype(bias_dtype)) || (residual && !known_dtype(residual_dtype)))
    return OPR_UNSUPPORTED;
  if (m == 0) return OPR_OK;
  if (!x || !w || !y || !dev_status || !words_aligned(dev_status)) return OPR_INVALID_ARG;
  if (!element_aligned(x, dtype) || !element_aligned(w, dtype) || !element_aligned(y, y_dtype) ||
      !element_aligned(z, dtype) || (bias && !element_aligned(bias, bias_dtype)) ||
      (residual && !element_aligned(residual, residual_dtype)))
    return OPR_INVALID_ARG;
  const size_t need = opr_linear_workspace_bytes(x, ldx, w, ldw, m, n, k);
  if (workspace_bytes < need) return OPR_WORKSPACE_TOO_SMALL;
  if (need > 0 && (!workspace || !aligned16(workspace))) return OPR_INVALID_ARG;
  const int64_t ws_words = static_cast<int64_t>(need / sizeof(float));
  const Rows in[4] = {{x, m, ldx, k, dtype},
                      {w, n, ldw, k, dtype},
                      {bias, 1, n, n, bias_dtype},
                      {residual, m, ld_residual, n, residual_dtype}};
  const OutRows out[3] = {{{y, m, ldy, n, y_dtype}, {&in[3], nullptr}},
                          {{z, m, ldz, n, dtype}, {nullptr, nullptr}},
                          {{workspace, 1, ws_words, ws_words, OPR_DTYPE_FP32}, {nullptr, nullptr}}};
  if (outputs_clash(in, out)) return OPR_INVALID_ARG;
  opr_status st = device_check();
  if (st != OPR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Operand ox{x, ldx, 1}, ow{w, ldw, 1};
  char* to = static_cast<char*>(workspace);
  PackJob jobs[2] = {};
  if (!tma_ready(x, ldx)) {
    jobs[0] = pack(ox, m, k, to);
    to += copy_bytes(m, k);
  }
  if (!tma_ready(w, ldw)) jobs[1] = pack(ow, n, k, to);
  st = status_of(launch_pack(jobs, s));
  if (st != OPR_OK) return st;
  LinearEpilogue e{bias, bias_dtype, activation, residual, ld_residual, residual_dtype, y, ldy, y_dtype, z, ldz};
  return status_of(launch_linear(ox, ow, m, n, k, dtype, e, dev_status, s));
}

namespace {
// Scratch of the gradients: dz (needed where it is not dy itself), copies of x
// and w with padded rows, and the partial column sums of dz.
struct LinearBwdWs {
  bool own_dz;
  size_t dz, x, w, partial, bytes;
};
LinearBwdWs linear_bwd_ws(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                          int64_t m, int32_t n, int32_t k, int32_t activation) {
  LinearBwdWs s{};
  s.own_dz = activation != OPR_ACT_NONE || !tma_ready(dy, ld_dy);
  s.x = s.own_dz ? copy_bytes(m, n) : 0;
  s.w = s.x + (tma_ready(x, ldx) ? 0 : copy_bytes(m, k));
  s.partial = s.w + (tma_ready(w, ldw) ? 0 : copy_bytes(n, k));
  s.bytes = s.partial + align_up(static_cast<size_t>(linear_dz_blocks(m, n)) * static_cast<size_t>(n) * sizeof(float), 256);
  return s;
}
}  // namespace

size_t opr_linear_bwd_workspace_bytes(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, const void* w,
                                      int64_t ldw, int64_t m, int32_t n, int32_t k, int32_t activation) {
  if (!linear_sizes_ok(m, n, k) || ld_dy < n || ldx < k || ldw < k || !known_act(activation)) return 0;
  return linear_bwd_ws(dy, ld_dy, x, ldx, w, ldw, m, n, k, activation).bytes;
}

opr_status opr_linear_bwd(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                          int32_t dtype, const void* z, int64_t ldz, int32_t activation, const void* dx_residual,
                          int64_t ld_residual, int32_t residual_dtype, void* dx, int64_t ld_dx, int32_t dx_dtype,
                          void* dw, int64_t ld_dw, int32_t dw_dtype, float* db, int64_t m, int32_t n, int32_t k,
                          void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  CallRange range("opr_linear_bwd");
  if (!linear_sizes_ok(m, n, k) || ld_dy < n || ldx < k || ldw < k) return OPR_INVALID_ARG;
  if (!known_act(activation)) return OPR_UNSUPPORTED;
  if (dtype != OPR_DTYPE_BF16 && dtype != OPR_DTYPE_FP16) return OPR_UNSUPPORTED;
  if ((dx && !known_dtype(dx_dtype)) || (dw && !known_dtype(dw_dtype)) ||
      (dx_residual && !known_dtype(residual_dtype)))
    return OPR_UNSUPPORTED;
  if ((dx && ld_dx < k) || (dw && ld_dw < k) || (dx_residual && ld_residual < k)) return OPR_INVALID_ARG;
  const bool act = activation != OPR_ACT_NONE;
  if (act && ldz < n) return OPR_INVALID_ARG;
  if (!dx && !dw && !db) return OPR_OK;
  if (m > 0 && (!dy || !x || !w || (act && !z))) return OPR_INVALID_ARG;
  if (!dev_status || !words_aligned(dev_status) || (dx_residual && !dx)) return OPR_INVALID_ARG;
  if (!element_aligned(dy, dtype) || !element_aligned(x, dtype) || !element_aligned(w, dtype) ||
      (act && !element_aligned(z, dtype)) || (dx && !element_aligned(dx, dx_dtype)) ||
      (dw && !element_aligned(dw, dw_dtype)) || !element_aligned(db, OPR_DTYPE_FP32) ||
      (dx_residual && !element_aligned(dx_residual, residual_dtype)))
    return OPR_INVALID_ARG;
  const LinearBwdWs ws = linear_bwd_ws(dy, ld_dy, x, ldx, w, ldw, m, n, k, activation);
  if (workspace_bytes < ws.bytes) return OPR_WORKSPACE_TOO_SMALL;
  if (ws.bytes > 0 && (!workspace || !aligned16(workspace))) return OPR_INVALID_ARG;
  const int64_t ws_words = static_cast<int64_t>(ws.bytes / sizeof(float));
  const Rows in[5] = {{dy, m, ld_dy, n, dtype},
                      {x, m, ldx, k, dtype},
                      {w, n, ldw, k, dtype},
                      {act ? z : nullptr, m, ldz, n, dtype},
                      {dx_residual, m, ld_residual, k, residual_dtype}};
  const OutRows out[4] = {{{dx, m, ld_dx, k, dx_dtype}, {&in[4], nullptr}},
                          {{dw, n, ld_dw, k, dw_dtype}, {nullptr, nullptr}},
                          {{db, 1, n, n, OPR_DTYPE_FP32}, {nullptr, nullptr}},
                          {{workspace, 1, ws_words, ws_words, OPR_DTYPE_FP32}, {nullptr, nullptr}}};
  if (outputs_clash(in, out)) return OPR_INVALID_ARG;
  opr_status st = device_check();
  if (st != OPR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* wsp = static_cast<char*>(workspace);
  const void* dz = dy;
  int64_t ld_dz = ld_dy;
  const bool own_dz = ws.own_dz && (dx || dw);
  if (own_dz) {
    dz = wsp + ws.dz;
    ld_dz = padded(n);
  }
  if (own_dz || db) {
    st = status_of(launch_linear_dz(dy, ld_dy, z, ldz, dtype, m, n, activation, own_dz ? wsp + ws.dz : nullptr, ld_dz,
                                    db, reinterpret_cast<float*>(wsp + ws.partial), dev_status, s));
    if (st != OPR_OK) return st;
  }
  Operand ox{x, ldx, 1}, ow{w, ldw, 1};
  PackJob jobs[2] = {};
  if (dw && m > 0 && !tma_ready(x, ldx)) jobs[0] = pack(ox, m, k, wsp + ws.x);
  if (dx && m > 0 && !tma_ready(w, ldw)) jobs[1] = pack(ow, n, k, wsp + ws.w);
  st = status_of(launch_pack(jobs, s));
  if (st != OPR_OK) return st;
  if (dx) {
    LinearEpilogue e{};
    e.residual = dx_residual;
    e.ld_residual = ld_residual;
    e.residual_dtype = residual_dtype;
    e.y = dx;
    e.ldy = ld_dx;
    e.y_dtype = dx_dtype;
    st = status_of(launch_linear(Operand{dz, ld_dz, 1}, Operand{ow.p, 1, ow.row}, m, k, n, dtype, e, dev_status, s));
    if (st != OPR_OK) return st;
  }
  if (dw) {
    LinearEpilogue e{};
    e.y = dw;
    e.ldy = ld_dw;
    e.y_dtype = dw_dtype;
    st = status_of(launch_linear(Operand{dz, 1, ld_dz}, Operand{ox.p, 1, ox.row}, n, k, m, dtype, e, dev_status, s));
  }
  return st;
}

}  // extern "C"
