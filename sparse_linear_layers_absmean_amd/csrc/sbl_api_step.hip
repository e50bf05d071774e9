// C ABI of the norm, the embedding and the AdamW update: host-side validation
// and dispatch.  See include/sbl.h.
#include <algorithm>
#include <cmath>
#include <new>

#include "sbl.h"
#include "sbl_host.h"
#include "sbl_step.h"

namespace {

using sbl::aligned;
using sbl::launch_status;
using sbl::ranges_overlap;
using sbl::step::type_bytes;

constexpr int64_t kMaxK = 131072;
constexpr int64_t kMaxTokens = int64_t(1) << 22;
constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr int64_t kMaxValues = int64_t(1) << 34;
constexpr int32_t kMaxItems = 65536;

static_assert((int)SBL_BF16 == sbl::step::kBf16 && (int)SBL_FP16 == sbl::step::kFp16 && (int)SBL_FP32 == sbl::step::kFp32,
              "types");

bool type_ok(int32_t t) { return t == SBL_BF16 || t == SBL_FP16 || t == SBL_FP32; }
// two types of one call: the same, or fp32 and any other
bool pair_ok(int32_t a, int32_t b) { return type_ok(a) && type_ok(b) && (a == b || a == SBL_FP32 || b == SBL_FP32); }

bool rows_ok(int64_t m_tok, int64_t k) {
  return m_tok >= 0 && m_tok <= kMaxTokens && k >= 1 && k <= kMaxK && m_tok * k <= kMaxValues;
}

struct Range {
  const void* p;
  int64_t bytes;
};

// whether one of the outputs shares a byte with another, or with an input
template <int NO, int NI> bool overlap(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
    for (const Range& r : in)
      if (ranges_overlap(out[i].p, out[i].bytes, r.p, r.bytes)) return true;
  }
  return false;
}

bool embed_ok(int64_t m_tok, int64_t n_vocab, int64_t k) {
  return rows_ok(m_tok, k) && n_vocab >= 1 && n_vocab <= kMaxVocab && n_vocab * k <= kMaxValues;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- norm

int sbl_norm_forward(const void* x, int32_t x_dtype, const float* weight, const float* bias, int64_t m_tok, int64_t k,
                     double eps, int32_t center, void* y, int32_t y_dtype, int8_t* xq, float* gamma, float* mean,
                     float* rstd, sbl_stream stream) {
  if (!rows_ok(m_tok, k) || !((float)eps > 0.0f) || !std::isfinite(eps)) return SBL_ERR_SHAPE;
  if (!pair_ok(x_dtype, y_dtype)) return SBL_ERR_UNSUPPORTED;
  if ((xq || gamma) && k % 64 != 0) return SBL_ERR_SHAPE;
  if (m_tok == 0) return SBL_OK;
  if (!x || !xq != !gamma) return SBL_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(xq, 16) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(gamma, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return SBL_ERR_ALIGN;
  const int64_t n = m_tok * k;
  const Range out[] = {{y, n * type_bytes(y_dtype)}, {xq, n}, {gamma, m_tok * 4}, {mean, m_tok * 4}, {rstd, m_tok * 4}};
  const Range in[] = {{x, n * type_bytes(x_dtype)}, {weight, k * 4}, {bias, k * 4}};
  if (overlap(out, in)) return SBL_ERR_SHAPE;
  if (!y && !xq && !mean && !rstd) return SBL_OK;
  const sbl::step::NormArgs a{x, weight, bias, m_tok, (int32_t)k, center != 0, eps, y, xq, gamma, mean, rstd};
  return launch_status(sbl::step::launch_norm_forward(a, x_dtype, y_dtype, reinterpret_cast<hipStream_t>(stream)));
}

int64_t sbl_norm_workspace_bytes(int64_t m_tok, int64_t k) {
  return rows_ok(m_tok, k) ? sbl::step::norm_grad_ws_bytes(m_tok, k) : -1;
}

int sbl_norm_backward(const void* dy, int32_t dy_dtype, const void* x, int32_t x_dtype, const float* mean,
                      const float* rstd, const float* weight, int64_t m_tok, int64_t k, int32_t center, void* dx,
                      float* dweight, float* dbias, void* workspace, int64_t workspace_bytes, sbl_stream stream) {
  if (!rows_ok(m_tok, k)) return SBL_ERR_SHAPE;
  if (!pair_ok(x_dtype, dy_dtype)) return SBL_ERR_UNSUPPORTED;
  const int64_t n = m_tok * k, need = sbl::step::norm_grad_ws_bytes(m_tok, k);
  if (m_tok > 0) {
    if (!dy || !x || !rstd || (center && !mean)) return SBL_ERR_NULL;
    if ((need > 0 && !workspace) || workspace_bytes < need) return SBL_ERR_WORKSPACE;
  }
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dx, 16) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(weight, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) || (m_tok > 0 && !aligned(workspace, 256)))
    return SBL_ERR_ALIGN;
  const Range out[] = {{dx, n * type_bytes(x_dtype)}, {dweight, k * 4}, {dbias, k * 4}, {m_tok > 0 ? workspace : nullptr, need}};
  const Range in[] = {{dy, n * type_bytes(dy_dtype)}, {x, n * type_bytes(x_dtype)}, {center ? mean : nullptr, m_tok * 4},
                      {rstd, m_tok * 4}, {weight, k * 4}};
  if (overlap(out, in)) return SBL_ERR_SHAPE;
  if (!dx && !dweight && !dbias) return SBL_OK;
  const sbl::step::NormGradArgs a{dy, x, center ? mean : nullptr, rstd, weight, m_tok, (int32_t)k, center != 0,
                                  dx, dweight, dbias, static_cast<float*>(workspace)};
  return launch_status(sbl::step::launch_norm_backward(a, x_dtype, dy_dtype, reinterpret_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- embedding

int sbl_embed_forward(const int64_t* ids, const void* table, int32_t table_dtype, int64_t m_tok, int64_t n_vocab,
                      int64_t k, float scale, void* out, int32_t out_dtype, sbl_stream stream) {
  if (!embed_ok(m_tok, n_vocab, k)) return SBL_ERR_SHAPE;
  if (!pair_ok(table_dtype, out_dtype)) return SBL_ERR_UNSUPPORTED;
  if (m_tok == 0) return SBL_OK;
  if (!ids || !table || !out) return SBL_ERR_NULL;
  if (!aligned(ids, 8) || !aligned(table, 16) || !aligned(out, 16)) return SBL_ERR_ALIGN;
  const Range o[] = {{out, m_tok * k * type_bytes(out_dtype)}};
  const Range in[] = {{ids, m_tok * 8}, {table, n_vocab * k * type_bytes(table_dtype)}};
  if (overlap(o, in)) return SBL_ERR_SHAPE;
  const sbl::step::EmbedArgs a{ids, table, m_tok, n_vocab, (int32_t)k, scale, out};
  return launch_status(sbl::step::launch_embed_forward(a, table_dtype, out_dtype, reinterpret_cast<hipStream_t>(stream)));
}

int64_t sbl_embed_workspace_bytes(int64_t m_tok, int64_t n_vocab, int64_t k, int32_t dout_dtype) {
  if (!embed_ok(m_tok, n_vocab, k) || !type_ok(dout_dtype)) return -1;
  return sbl::step::embed_grad_ws_bytes(m_tok, n_vocab, k, dout_dtype);
}

int sbl_embed_backward(const int64_t* ids, const void* dout, int32_t dout_dtype, int64_t m_tok, int64_t n_vocab,
                       int64_t k, float scale, void* dtable, int32_t table_dtype, int32_t add, void* workspace,
                       int64_t workspace_bytes, sbl_stream stream) {
  if (!embed_ok(m_tok, n_vocab, k)) return SBL_ERR_SHAPE;
  if (!pair_ok(table_dtype, dout_dtype)) return SBL_ERR_UNSUPPORTED;
  if (m_tok == 0 && add) return SBL_OK;
  if (!dtable || (m_tok > 0 && (!ids || !dout))) return SBL_ERR_NULL;
  const int64_t need = sbl::step::embed_grad_ws_bytes(m_tok, n_vocab, k, dout_dtype);
  if (!workspace || workspace_bytes < need) return SBL_ERR_WORKSPACE;
  if (!aligned(ids, 8) || !aligned(dout, 16) || !aligned(dtable, 16) || !aligned(workspace, 256)) return SBL_ERR_ALIGN;
  const Range out[] = {{dtable, n_vocab * k * type_bytes(table_dtype)}, {workspace, need}};
  const Range in[] = {{ids, m_tok * 8}, {dout, m_tok * k * type_bytes(dout_dtype)}};
  if (overlap(out, in)) return SBL_ERR_SHAPE;
  const sbl::step::EmbedGradArgs a{ids, dout, m_tok, n_vocab, (int32_t)k, scale, dtable, add != 0, workspace};
  return launch_status(sbl::step::launch_embed_backward(a, dout_dtype, table_dtype, reinterpret_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- AdamW

namespace {

// every buffer of an item; those that are written first
constexpr int kItemWritten = 6, kItemBuffers = 7;

void item_ranges(const sbl_adamw_item& it, Range (&r)[kItemBuffers]) {
  const bool small = it.state_bits == 8;
  const int64_t state = it.n * (small ? 1 : 4), scales = small ? (it.n + 255) / 256 * 4 : 0;
  r[0] = Range{it.w, it.n * type_bytes(it.w_dtype)};
  r[1] = Range{it.w_low, it.n * 2};
  r[2] = Range{it.m, state};
  r[3] = Range{it.v, state};
  r[4] = Range{small ? it.m_scale : nullptr, scales};
  r[5] = Range{small ? it.v_scale : nullptr, scales};
  r[6] = Range{it.g, it.n * type_bytes(it.g_dtype)};
}

int check_adamw(const sbl_adamw_item& it) {
  if (it.n < 0 || it.n > kMaxValues || !std::isfinite(it.lr_scale) || !std::isfinite(it.weight_decay)) return SBL_ERR_SHAPE;
  if (!type_ok(it.w_dtype) || !type_ok(it.g_dtype) || (it.state_bits != 8 && it.state_bits != 32) ||
      (it.w_low && it.w_dtype != SBL_BF16))
    return SBL_ERR_UNSUPPORTED;
  if (it.n == 0) return SBL_OK;
  if (!it.w || !it.g || !it.m || !it.v || (it.state_bits == 8 && (!it.m_scale || !it.v_scale))) return SBL_ERR_NULL;
  const uintptr_t state = it.state_bits == 8 ? 8 : 4;
  if (!aligned(it.w, (uintptr_t)type_bytes(it.w_dtype)) || !aligned(it.w_low, 2) ||
      !aligned(it.g, (uintptr_t)type_bytes(it.g_dtype)) || !aligned(it.m, state) || !aligned(it.v, state) ||
      (it.state_bits == 8 && (!aligned(it.m_scale, 4) || !aligned(it.v_scale, 4))))
    return SBL_ERR_ALIGN;
  return SBL_OK;
}

struct Span {
  uintptr_t begin, end;
  bool written;
};

// Whether a written buffer shares a byte with any other: in order of their
// addresses, one that begins before an earlier one ends, one of the two written.
bool spans_collide(Span* s, int64_t n) {
  std::sort(s, s + n, [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any = 0, written = 0;                // furthest ends so far
  for (int64_t i = 0; i < n; ++i) {
    if (s[i].begin < written || (s[i].written && s[i].begin < any)) return true;
    any = std::max(any, s[i].end);
    if (s[i].written) written = std::max(written, s[i].end);
  }
  return false;
}

}  // namespace

int sbl_adamw_batch(const sbl_adamw_item* items, int32_t count, double lr, double beta1, double beta2, double eps,
                    int64_t step, const float* schedule, sbl_stream stream) {
  if (count < 1 || count > kMaxItems) return SBL_ERR_SHAPE;
  if (!items) return SBL_ERR_NULL;
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0) || !((float)eps > 0.0f) || !std::isfinite((float)eps))
    return SBL_ERR_SHAPE;
  if (!schedule && (step < 1 || !std::isfinite((float)lr))) return SBL_ERR_SHAPE;
  for (int32_t i = 0; i < count; ++i) {
    const int st = check_adamw(items[i]);
    if (st != SBL_OK) return st;
  }
  if (!aligned(schedule, 4)) return SBL_ERR_ALIGN;
  const int64_t most = (int64_t)count * kItemBuffers + 1;
  Span* spans = new (std::nothrow) Span[most];
  sbl::step::AdamItem* to = new (std::nothrow) sbl::step::AdamItem[count];
  int64_t n = 0;
  if (spans && schedule) spans[n++] = Span{reinterpret_cast<uintptr_t>(schedule), reinterpret_cast<uintptr_t>(schedule + 5), false};
  for (int32_t i = 0; spans && to && i < count; ++i) {
    const sbl_adamw_item& it = items[i];
    Range r[kItemBuffers];
    item_ranges(it, r);
    for (int j = 0; j < kItemBuffers; ++j)
      if (r[j].p && r[j].bytes > 0)
        spans[n++] = Span{reinterpret_cast<uintptr_t>(r[j].p), reinterpret_cast<uintptr_t>(r[j].p) + (uintptr_t)r[j].bytes,
                          j < kItemWritten};
    to[i] = sbl::step::AdamItem{it.w, it.w_low, it.g, it.m, it.v, it.m_scale, it.v_scale, it.n, it.lr_scale,
                                it.weight_decay, it.w_dtype + 3 * it.g_dtype, it.state_bits};
  }
  int status = SBL_ERR_WORKSPACE;                // no host memory for the lists
  if (spans && to) {
    if (spans_collide(spans, n)) {
      status = SBL_ERR_SHAPE;
    } else {
      sbl::step::AdamStep s{};
      s.b1 = (float)beta1;
      s.a1 = (float)(1.0 - beta1);
      s.b2 = (float)beta2;
      s.a2 = (float)(1.0 - beta2);
      s.eps = (float)eps;
      s.schedule = reinterpret_cast<const sbl::step::AdamSchedule*>(schedule);
      if (!schedule)
        s.now = sbl::step::AdamSchedule{(float)lr, (float)(1.0 / (1.0 - std::pow(beta1, (double)step))),
                                        (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step))), 1.0f,
                                        (float)(step % (1 << 24))};
      status = launch_status(sbl::step::launch_adamw(to, count, s, reinterpret_cast<hipStream_t>(stream)));
    }
  }
  delete[] spans;
  delete[] to;
  return status;
}

}  // extern "C"
