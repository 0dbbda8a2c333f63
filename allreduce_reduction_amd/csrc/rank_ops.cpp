// C entry points of the row operators over the ranks: argument checks and
// launches (kernels in norm_kernels.hip, embedding_kernels.hip and
// distill_kernels.hip).
#include <algorithm>
#include <vector>

#include "comm.hpp"
#include "hbmcoll.h"
#include "rowops.hpp"

using namespace hbmc;

namespace {

// Memory ranges of a call.  A range that is written may overlap no other;
// ranges that are only read may overlap each other.
class Ranges {
 public:
  // [p, p + bytes), checked for NULL, alignment and wrap-around; nothing to
  // check where it holds nothing.
  void add(const void* p, uint64_t bytes, uint32_t align, bool write) {
    if (bytes == 0) return;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (!a || a % align || a + bytes < a) bad_ = true;
    all_.push_back({a, a + bytes, write});
  }
  void read(const void* p, uint64_t bytes, uint32_t align) { add(p, bytes, align, false); }
  void write(const void* p, uint64_t bytes, uint32_t align) { add(p, bytes, align, true); }
  // An output that may be exactly the input `in`, which is then not added.
  void write_over(const void* p, const void* in, uint64_t bytes, uint32_t align) {
    write(p, bytes, align);
    if (in != p) read(in, bytes, align);
  }
  bool ok() {
    if (bad_) return false;
    std::sort(all_.begin(), all_.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
    uintptr_t any = 0, written = 0;  // ends of the ranges so far, of the written ones
    for (const Range& r : all_) {
      if (r.lo < written || (r.write && r.lo < any)) return false;
      any = std::max(any, r.hi);
      if (r.write) written = std::max(written, r.hi);
    }
    return true;
  }

 private:
  struct Range {
    uintptr_t lo, hi;
    bool write;
  };
  std::vector<Range> all_;
  bool bad_ = false;
};

// Element size of a type the operators take (0: they do not).
uint32_t float_bytes(int dtype) { return dtype == HBMC_FP32 || dtype == HBMC_FP16 || dtype == HBMC_BF16 ? elem_bytes(dtype) : 0; }

bool finite(float x) { return x - x == 0.0f; }

constexpr uint64_t kMaxRows = (uint64_t(1) << 31) - 1;

int ranks_of(hbmc_comm_t c) { return c && !c->topos.empty() ? c->topos[0].P : 0; }

// Bytes of a matrix, or false when they do not fit an address.
bool matrix_bytes(uint64_t rows, uint64_t width, uint32_t e, uint64_t* bytes) {
  return !__builtin_mul_overflow(rows, width, bytes) && !__builtin_mul_overflow(*bytes, uint64_t(e), bytes) &&
         *bytes <= uint64_t(PTRDIFF_MAX);
}

hbmc_status_t hip(hipError_t e) { return e == hipSuccess ? HBMC_OK : HBMC_ERR_HIP; }

// ------------------------------------------------------------------ norms

hbmc_status_t norm_shape(hbmc_comm_t comm, const hbmc_norm_t* n, NormShape* s) {
  const int P = ranks_of(comm);
  if (P == 0 || !n || float_bytes(n->dtype) == 0 || n->width == 0 || n->rows > kMaxRows) {
    const bool known = P > 0 && n && (n->dtype == HBMC_INT32 || n->dtype == HBMC_INT8);
    return known ? HBMC_ERR_UNSUPPORTED : HBMC_ERR_INVALID_ARG;
  }
  if (n->width > kNormMaxWidth) return HBMC_ERR_UNSUPPORTED;
  uint64_t bytes;
  if (!matrix_bytes(n->rows, n->width, 4, &bytes)) return HBMC_ERR_INVALID_ARG;
  if (!finite(n->scale) || !finite(n->pre_eps) || n->pre_eps < 0 || (n->post_weight && (!finite(n->post_eps) || n->post_eps < 0)))
    return HBMC_ERR_INVALID_ARG;
  if (!n->pre_weight || (n->gate && n->gate_rows == 0)) return HBMC_ERR_INVALID_ARG;
  const uint64_t rows = std::max<uint64_t>(n->rows, 1);
  s->rows = static_cast<uint32_t>(n->rows);
  s->seg = static_cast<uint32_t>(segment_each(rows, P));
  s->width = static_cast<uint32_t>(n->width);
  s->gate_rows = static_cast<uint32_t>(n->gate ? std::min<uint64_t>(n->gate_rows, rows) : rows);
  s->P = P;
  s->scale = n->scale;
  s->pre_eps = n->pre_eps;
  s->post_eps = n->post_eps;
  s->pre_weight = n->pre_weight;
  s->post_weight = n->post_weight;
  s->gate = n->gate;
  return HBMC_OK;
}

void read_weights(const NormShape& s, uint32_t e, Ranges* r) {
  const uint64_t row = uint64_t(s.width) * e;
  r->read(s.pre_weight, row, e);
  if (s.post_weight) r->read(s.post_weight, row, e);
  if (s.gate && s.rows > 0) r->read(s.gate, ((s.rows - 1) / s.gate_rows + 1) * row, e);
}

hbmc_status_t reduce_norm(hbmc_comm_t comm, const hbmc_norm_t* norm, const void* const parts[], const void* const residual[],
                          void* const residual_out[], void* const out[], void* const sums[], void* stream) {
  NormShape s;
  hbmc_status_t st = norm_shape(comm, norm, &s);
  if (st != HBMC_OK) return st;
  if (!parts || !residual || !residual_out || !out) return HBMC_ERR_INVALID_ARG;
  const uint32_t e = float_bytes(norm->dtype);
  const uint64_t row = uint64_t(s.width) * e;
  NormPtrs a = {};
  a.save = sums != nullptr;
  Ranges r;
  read_weights(s, e, &r);
  for (int p = 0; p < s.P; ++p) {
    a.parts[p] = static_cast<const unsigned char*>(parts[p]);
    a.out[p] = static_cast<unsigned char*>(out[p]);
    r.write_over(out[p], parts[p], s.rows * row, e);
    const uint64_t mine = segment_count(s.rows, s.P, p) * row;
    a.residual[p] = static_cast<const unsigned char*>(residual[p]);
    a.residual_out[p] = static_cast<unsigned char*>(residual_out[p]);
    r.write_over(residual_out[p], residual[p], mine, e);
    if (sums) {
      a.sums[p] = static_cast<unsigned char*>(sums[p]);
      r.write(sums[p], mine, e);
    }
  }
  if (!r.ok()) return HBMC_ERR_INVALID_ARG;
  if (s.rows == 0) return HBMC_OK;
  return hip(launch_norm(norm->dtype, a, s, static_cast<hipStream_t>(stream)));
}

hbmc_status_t reduce_norm_grad(hbmc_comm_t comm, const hbmc_norm_t* norm, const void* const out_grads[],
                               const void* const hidden[], const void* const sums[], const void* const residual_grad_in[],
                               void* const part_grads[], void* const residual_grad[], float* pre_weight_grad,
                               float* post_weight_grad, float* gate_grad, void* workspace, size_t workspace_bytes,
                               void* stream) {
  NormShape s;
  hbmc_status_t st = norm_shape(comm, norm, &s);
  if (st != HBMC_OK) return st;
  const bool has_sum = s.post_weight || s.gate;
  if (!out_grads || !hidden || !part_grads || !residual_grad || !pre_weight_grad || (has_sum && !sums) ||
      (s.post_weight && !post_weight_grad) || (!s.post_weight && post_weight_grad) || (!s.gate && gate_grad) ||
      (s.gate && s.rows > 0 && !gate_grad))
    return HBMC_ERR_INVALID_ARG;
  const NormGradSplit d = split_norm_grad(norm->dtype, s);
  if (workspace_bytes < d.bytes) return HBMC_ERR_INVALID_ARG;
  const uint32_t e = float_bytes(norm->dtype);
  const uint64_t row = uint64_t(s.width) * e, wide = uint64_t(s.width) * 4;
  NormGradPtrs a = {};
  a.has_in = residual_grad_in != nullptr;
  a.partial = static_cast<float*>(workspace);
  Ranges r;
  read_weights(s, e, &r);
  for (int p = 0; p < s.P; ++p) {
    a.out_grads[p] = static_cast<const unsigned char*>(out_grads[p]);
    a.part_grads[p] = static_cast<unsigned char*>(part_grads[p]);
    r.write_over(part_grads[p], out_grads[p], s.rows * row, e);
    const uint64_t mine = segment_count(s.rows, s.P, p) * row;
    a.hidden[p] = static_cast<const unsigned char*>(hidden[p]);
    r.read(hidden[p], mine, e);
    if (has_sum) {
      a.sums[p] = static_cast<const unsigned char*>(sums[p]);
      r.read(sums[p], mine, e);
    }
    a.residual_out[p] = static_cast<unsigned char*>(residual_grad[p]);
    if (a.has_in) {
      a.residual_in[p] = static_cast<const unsigned char*>(residual_grad_in[p]);
      r.write_over(residual_grad[p], residual_grad_in[p], mine, e);
    } else {
      r.write(residual_grad[p], mine, e);
    }
  }
  r.write(pre_weight_grad, wide, 4);
  if (s.post_weight) r.write(post_weight_grad, wide, 4);
  if (s.gate) r.write(gate_grad, d.groups * wide, 4);
  r.write(workspace, d.bytes, 16);
  if (!r.ok()) return HBMC_ERR_INVALID_ARG;
  return hip(launch_norm_grad(norm->dtype, a, s, d, pre_weight_grad, post_weight_grad, gate_grad,
                              static_cast<hipStream_t>(stream)));
}

// -------------------------------------------------------------- embedding

hbmc_status_t embed_args(hbmc_comm_t comm, const hbmc_embedding_t* m, const size_t tokens[], EmbedArgs* a, uint64_t* total) {
  const int P = ranks_of(comm);
  if (P == 0 || !m || !tokens) return HBMC_ERR_INVALID_ARG;
  if (float_bytes(m->dtype) == 0)
    return m->dtype == HBMC_INT32 || m->dtype == HBMC_INT8 ? HBMC_ERR_UNSUPPORTED : HBMC_ERR_INVALID_ARG;
  uint64_t bytes;
  if (m->vocab == 0 || m->vocab > kMaxVocab || m->width == 0 || m->width > (uint64_t(1) << 24) || !finite(m->scale) ||
      (m->id_bytes != 4 && m->id_bytes != 8) || !matrix_bytes(m->vocab, m->width, 4, &bytes))
    return HBMC_ERR_INVALID_ARG;
  *total = 0;
  for (int p = 0; p < P; ++p) {
    if (tokens[p] >= kMaxTokens) return HBMC_ERR_INVALID_ARG;
    a->tokens[p] = static_cast<uint32_t>(tokens[p]);
    *total += tokens[p];
  }
  if (*total > kMaxRows) return HBMC_ERR_INVALID_ARG;
  a->seg = static_cast<uint32_t>(segment_each(m->vocab, P));
  a->vocab = static_cast<uint32_t>(m->vocab);
  a->width = static_cast<uint32_t>(m->width);
  a->P = P;
  a->id_bytes = m->id_bytes;
  a->scale = m->scale;
  return HBMC_OK;
}

hbmc_status_t embedding(hbmc_comm_t comm, const hbmc_embedding_t* m, const void* const tables[], const void* const ids[],
                        const size_t tokens[], void* const out[], void* stream) {
  EmbedArgs a = {};
  uint64_t total;
  hbmc_status_t st = embed_args(comm, m, tokens, &a, &total);
  if (st != HBMC_OK) return st;
  if (!tables || !ids || !out) return HBMC_ERR_INVALID_ARG;
  const uint32_t e = float_bytes(m->dtype);
  const uint64_t row = uint64_t(a.width) * e;
  Ranges r;
  for (int p = 0; p < a.P; ++p) {
    a.rows[p] = static_cast<const unsigned char*>(tables[p]);
    a.ids[p] = static_cast<const unsigned char*>(ids[p]);
    a.out[p] = static_cast<unsigned char*>(out[p]);
    r.read(tables[p], segment_count(a.vocab, a.P, p) * row, e);
    r.read(ids[p], uint64_t(a.tokens[p]) * a.id_bytes, a.id_bytes);
    r.write(out[p], a.tokens[p] * row, e);
  }
  if (!r.ok()) return HBMC_ERR_INVALID_ARG;
  if (total == 0) return HBMC_OK;
  return hip(launch_embed(m->dtype, a, static_cast<hipStream_t>(stream)));
}

hbmc_status_t embedding_grad(hbmc_comm_t comm, const hbmc_embedding_t* m, const void* const out_grads[], const void* const ids[],
                             const size_t tokens[], void* const table_grads[], hbmc_dtype_t grad_dtype, int accumulate,
                             void* workspace, size_t workspace_bytes, void* stream) {
  EmbedArgs a = {};
  uint64_t total;
  hbmc_status_t st = embed_args(comm, m, tokens, &a, &total);
  if (st != HBMC_OK) return st;
  if (!out_grads || !ids || !table_grads || (grad_dtype != HBMC_FP32 && grad_dtype != m->dtype)) return HBMC_ERR_INVALID_ARG;
  if (!embed_grad_fits(m->dtype, total, a.width)) return HBMC_ERR_UNSUPPORTED;
  const EmbedGradSplit d = split_embed_grad(m->dtype, total, a.vocab, a.width);
  if (workspace_bytes < d.bytes) return HBMC_ERR_INVALID_ARG;
  const uint32_t e = float_bytes(m->dtype), ge = float_bytes(grad_dtype);
  Ranges r;
  for (int p = 0; p < a.P; ++p) {
    a.rows[p] = static_cast<const unsigned char*>(out_grads[p]);
    a.ids[p] = static_cast<const unsigned char*>(ids[p]);
    a.out[p] = static_cast<unsigned char*>(table_grads[p]);
    r.read(out_grads[p], uint64_t(a.tokens[p]) * a.width * e, e);
    r.read(ids[p], uint64_t(a.tokens[p]) * a.id_bytes, a.id_bytes);
    r.write(table_grads[p], segment_count(a.vocab, a.P, p) * a.width * ge, ge);
  }
  r.write(workspace, d.bytes, 16);
  if (!r.ok()) return HBMC_ERR_INVALID_ARG;
  return hip(launch_embed_grad(m->dtype, grad_dtype, a, d, accumulate != 0, static_cast<unsigned char*>(workspace),
                               static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------ distillation

hbmc_status_t distill_args(hbmc_comm_t comm, const hbmc_distill_t* m, bool grad, DistillArgs* a) {
  const int P = ranks_of(comm);
  if (P == 0 || !m) return HBMC_ERR_INVALID_ARG;
  for (const int t : {static_cast<int>(m->dtype), static_cast<int>(m->teacher_dtype)})
    if (float_bytes(t) == 0) return t == HBMC_INT32 || t == HBMC_INT8 ? HBMC_ERR_UNSUPPORTED : HBMC_ERR_INVALID_ARG;
  uint64_t bytes;
  if (m->vocab == 0 || m->vocab > kMaxVocab || m->top == 0 || m->rows > kMaxRows || (m->id_bytes != 4 && m->id_bytes != 8) ||
      !(m->temperature > 0.0f) || !finite(1.0f / m->temperature * kLog2e) || !finite(m->temperature * m->temperature) ||
      !matrix_bytes(m->rows, m->vocab, 4, &bytes) || !matrix_bytes(m->rows, m->top, 8, &bytes))
    return HBMC_ERR_INVALID_ARG;
  if (m->top > kMaxTop) return HBMC_ERR_UNSUPPORTED;
  a->rows = m->rows;
  a->vocab = static_cast<uint32_t>(m->vocab);
  a->seg = static_cast<uint32_t>(segment_each(m->vocab, P));
  a->top = static_cast<uint32_t>(m->top);
  a->P = P;
  a->teacher_dtype = m->teacher_dtype;
  a->id_bytes = m->id_bytes;
  a->temperature = m->temperature;
  a->teacher = static_cast<const unsigned char*>(m->teacher_logits);
  a->ids = static_cast<const unsigned char*>(m->teacher_ids);
  a->pieces = distill_pieces(m->dtype, grad, a->seg);
  a->parts = a->pieces * static_cast<uint32_t>(P);
  if (a->rows * a->pieces > UINT32_MAX - 4) return HBMC_ERR_UNSUPPORTED;  // far past any memory
  return HBMC_OK;
}

void read_teacher(const DistillArgs& a, Ranges* r) {
  const uint32_t te = float_bytes(a.teacher_dtype);
  r->read(a.teacher, a.rows * a.top * te, te);
  r->read(a.ids, a.rows * a.top * a.id_bytes, a.id_bytes);
}

hbmc_status_t distill_loss(hbmc_comm_t comm, const hbmc_distill_t* m, const void* const logits[], float* loss, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  DistillArgs a = {};
  hbmc_status_t st = distill_args(comm, m, false, &a);
  if (st != HBMC_OK) return st;
  const uint64_t bytes = distill_workspace(m->dtype, a);
  if (!logits || workspace_bytes < bytes) return HBMC_ERR_INVALID_ARG;
  const uint32_t e = float_bytes(m->dtype);
  Ranges r;
  read_teacher(a, &r);
  for (int p = 0; p < a.P; ++p) {
    a.logits[p] = static_cast<const unsigned char*>(logits[p]);
    r.read(logits[p], a.rows * segment_count(a.vocab, a.P, p) * e, e);
  }
  r.write(loss, a.rows * 4, 4);
  r.write(lse, a.rows * 4, 4);
  r.write(workspace, bytes, 16);
  if (!r.ok()) return HBMC_ERR_INVALID_ARG;
  if (a.rows == 0) return HBMC_OK;
  a.loss = loss;
  a.lse = lse;
  a.partial = static_cast<float2*>(workspace);
  return hip(launch_distill(m->dtype, a, static_cast<hipStream_t>(stream)));
}

hbmc_status_t distill_loss_grad(hbmc_comm_t comm, const hbmc_distill_t* m, const void* const logits[], const float* lse,
                                const float* loss_grad, void* const logit_grads[], void* stream) {
  DistillArgs a = {};
  hbmc_status_t st = distill_args(comm, m, true, &a);
  if (st != HBMC_OK) return st;
  if (!logits || !logit_grads) return HBMC_ERR_INVALID_ARG;
  const uint32_t e = float_bytes(m->dtype);
  Ranges r;
  read_teacher(a, &r);
  for (int p = 0; p < a.P; ++p) {
    a.logits[p] = static_cast<const unsigned char*>(logits[p]);
    a.grads[p] = static_cast<unsigned char*>(logit_grads[p]);
    r.write_over(logit_grads[p], logits[p], a.rows * segment_count(a.vocab, a.P, p) * e, e);
  }
  r.read(lse, a.rows * 4, 4);
  r.read(loss_grad, a.rows * 4, 4);
  if (!r.ok()) return HBMC_ERR_INVALID_ARG;
  if (a.rows == 0) return HBMC_OK;
  a.lse = const_cast<float*>(lse);
  a.loss_grad = loss_grad;
  return hip(launch_distill_grad(m->dtype, a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

hbmc_status_t hbmc_reduce_norm(hbmc_comm_t comm, const hbmc_norm_t* norm, const void* const parts[], const void* const residual[],
                               void* const residual_out[], void* const out[], void* const sums[], void* stream) {
  return no_throw([&] { return reduce_norm(comm, norm, parts, residual, residual_out, out, sums, stream); });
}

hbmc_status_t hbmc_reduce_norm_grad_workspace(hbmc_comm_t comm, const hbmc_norm_t* norm, size_t* bytes) {
  return no_throw([&]() -> hbmc_status_t {
    NormShape s;
    if (!bytes) return HBMC_ERR_INVALID_ARG;
    const hbmc_status_t st = norm_shape(comm, norm, &s);
    if (st == HBMC_OK) *bytes = split_norm_grad(norm->dtype, s).bytes;
    return st;
  });
}

hbmc_status_t hbmc_reduce_norm_grad(hbmc_comm_t comm, const hbmc_norm_t* norm, const void* const out_grads[],
                                    const void* const hidden[], const void* const sums[], const void* const residual_grad_in[],
                                    void* const part_grads[], void* const residual_grad[], float* pre_weight_grad,
                                    float* post_weight_grad, float* gate_grad, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  return no_throw([&] {
    return reduce_norm_grad(comm, norm, out_grads, hidden, sums, residual_grad_in, part_grads, residual_grad, pre_weight_grad,
                            post_weight_grad, gate_grad, workspace, workspace_bytes, stream);
  });
}

hbmc_status_t hbmc_embedding(hbmc_comm_t comm, const hbmc_embedding_t* emb, const void* const tables[], const void* const ids[],
                             const size_t tokens[], void* const out[], void* stream) {
  return no_throw([&] { return embedding(comm, emb, tables, ids, tokens, out, stream); });
}

hbmc_status_t hbmc_embedding_grad_workspace(hbmc_comm_t comm, const hbmc_embedding_t* emb, const size_t tokens[], size_t* bytes) {
  return no_throw([&]() -> hbmc_status_t {
    EmbedArgs a = {};
    uint64_t total;
    if (!bytes) return HBMC_ERR_INVALID_ARG;
    const hbmc_status_t st = embed_args(comm, emb, tokens, &a, &total);
    if (st != HBMC_OK) return st;
    if (!embed_grad_fits(emb->dtype, total, a.width)) return HBMC_ERR_UNSUPPORTED;
    *bytes = split_embed_grad(emb->dtype, total, a.vocab, a.width).bytes;
    return HBMC_OK;
  });
}

hbmc_status_t hbmc_embedding_grad(hbmc_comm_t comm, const hbmc_embedding_t* emb, const void* const out_grads[],
                                  const void* const ids[], const size_t tokens[], void* const table_grads[],
                                  hbmc_dtype_t grad_dtype, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  return no_throw([&] {
    return embedding_grad(comm, emb, out_grads, ids, tokens, table_grads, grad_dtype, accumulate, workspace, workspace_bytes,
                          stream);
  });
}

hbmc_status_t hbmc_distill_loss_workspace(hbmc_comm_t comm, const hbmc_distill_t* distill, size_t* bytes) {
  return no_throw([&]() -> hbmc_status_t {
    DistillArgs a = {};
    if (!bytes) return HBMC_ERR_INVALID_ARG;
    const hbmc_status_t st = distill_args(comm, distill, false, &a);
    if (st == HBMC_OK) *bytes = distill_workspace(distill->dtype, a);
    return st;
  });
}

hbmc_status_t hbmc_distill_loss(hbmc_comm_t comm, const hbmc_distill_t* distill, const void* const logits[], float* loss,
                                float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return no_throw([&] { return distill_loss(comm, distill, logits, loss, lse, workspace, workspace_bytes, stream); });
}

hbmc_status_t hbmc_distill_loss_grad(hbmc_comm_t comm, const hbmc_distill_t* distill, const void* const logits[],
                                     const float* lse, const float* loss_grad, void* const logit_grads[], void* stream) {
  return no_throw([&] { return distill_loss_grad(comm, distill, logits, lse, loss_grad, logit_grads, stream); });
}

}  // extern "C"
