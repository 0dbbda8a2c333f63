// Gradient tensors of a training step: the handle that keeps their table on the
// device, and its calls (kernels in gradient_kernels.hip).
#include <hip/hip_runtime.h>

#include <cmath>
#include <new>
#include <vector>

#include "comm.hpp"
#include "hbmcoll.h"
#include "rank_args.hpp"
#include "rowops.hpp"

using namespace hbmc;

struct hbmc_gradients {
  int device = -1;
  uint32_t pieces = 0;
  uint64_t read = 0, written = 0;  // bytes of the tensors, of all their copies
  std::vector<std::pair<uintptr_t, uintptr_t>> held;  // the gradients' memory, ascending
  void* table = nullptr;
  const GradPiece* piece = nullptr;
  unsigned char* const* others = nullptr;
  ~hbmc_gradients() {
    if (table) (void)hipFree(table);
  }
};

namespace {

hbmc_status_t create(hbmc_comm_t comm, size_t n, const hbmc_gradient_t t[], hbmc_gradients* g) {
  const int P = ranks_of(comm);
  if (P == 0 || (n > 0 && !t)) return HBMC_ERR_INVALID_ARG;
  std::vector<GradPiece> pieces;
  std::vector<unsigned char*> others;
  Ranges r;
  for (size_t i = 0; i < n; ++i) {
    const uint32_t e = float_bytes(t[i].dtype);
    if (e == 0) return t[i].dtype == HBMC_INT32 || t[i].dtype == HBMC_INT8 ? HBMC_ERR_UNSUPPORTED : HBMC_ERR_INVALID_ARG;
    uint64_t bytes;
    if ((t[i].copies != 1 && t[i].copies != P) || !t[i].data || !matrix_bytes(t[i].count, 1, e, &bytes)) return HBMC_ERR_INVALID_ARG;
    if (bytes == 0) continue;
    for (int c = 0; c < t[i].copies; ++c) {
      r.write(t[i].data[c], bytes, e);
      const uintptr_t at = reinterpret_cast<uintptr_t>(t[i].data[c]);
      g->held.emplace_back(at, at + bytes);
    }
    if (r.bad()) return HBMC_ERR_INVALID_ARG;
    g->read += bytes;
    g->written += bytes * static_cast<uint64_t>(t[i].copies);
    GradPiece p = {};
    p.dtype = static_cast<uint32_t>(t[i].dtype);
    p.copies = static_cast<uint16_t>(t[i].copies);
    for (int c = 1; c < t[i].copies; ++c)
      if ((reinterpret_cast<uintptr_t>(t[i].data[c]) ^ reinterpret_cast<uintptr_t>(t[i].data[0])) & 127) p.shifted = 1;
    p.first = static_cast<uint32_t>(others.size());
    if (others.size() + static_cast<size_t>(P) > UINT32_MAX) return HBMC_ERR_UNSUPPORTED;
    for (int c = 1; c < t[i].copies; ++c) others.push_back(static_cast<unsigned char*>(t[i].data[c]));
    // the first piece ends where the tensor's address is a multiple of 256, so
    // that the others' vectors are aligned
    unsigned char* const base = static_cast<unsigned char*>(t[i].data[0]);
    uint64_t at = 0, most = kGradPieceBytes - reinterpret_cast<uintptr_t>(base) % 256;
    const uint64_t more = bytes > most ? 1 + (bytes - most + kGradPieceBytes - 1) / kGradPieceBytes : 1;
    if (more > kMaxGradPieces - pieces.size()) return HBMC_ERR_UNSUPPORTED;  // before a table of any length is made
    while (at < bytes) {
      const uint64_t here = std::min(most, bytes - at);
      p.data = base + at;
      p.offset = at;
      p.count = static_cast<uint32_t>(here / e);
      pieces.push_back(p);
      at += here;
      most = kGradPieceBytes;
    }
  }
  if (!r.ok()) return HBMC_ERR_INVALID_ARG;
  std::sort(g->held.begin(), g->held.end());
  g->pieces = static_cast<uint32_t>(pieces.size());
  if (hipGetDevice(&g->device) != hipSuccess) return HBMC_ERR_HIP;
  if (pieces.empty()) return HBMC_OK;
  const size_t a = pieces.size() * sizeof(GradPiece), b = others.size() * sizeof(unsigned char*);
  if (hipMalloc(&g->table, a + b) != hipSuccess) {
    g->table = nullptr;
    (void)hipGetLastError();
    return HBMC_ERR_NOMEM;
  }
  unsigned char* const base = static_cast<unsigned char*>(g->table);
  if (hipMemcpy(base, pieces.data(), a, hipMemcpyHostToDevice) != hipSuccess ||
      (b > 0 && hipMemcpy(base + a, others.data(), b, hipMemcpyHostToDevice) != hipSuccess))
    return HBMC_ERR_HIP;
  g->piece = reinterpret_cast<const GradPiece*>(base);
  g->others = reinterpret_cast<unsigned char* const*>(base + a);
  return HBMC_OK;
}

// Bytes of the partial sums and the factor.
uint64_t workspace_of(const hbmc_gradients* g) {
  const uint32_t sums = grad_sums(g->pieces, g->written);
  return sums ? (uint64_t(sums) + 1) * sizeof(double) : 0;
}

// Whether [p, p + bytes) is apart from every gradient.
bool apart(const hbmc_gradients* g, const void* p, uint64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + bytes;
  const auto next = std::upper_bound(g->held.begin(), g->held.end(), std::make_pair(lo, UINTPTR_MAX));
  if (next != g->held.end() && next->first < hi) return false;
  return next == g->held.begin() || std::prev(next)->second <= lo;
}

hbmc_status_t run(const hbmc_gradients* g, double norm_type, double scale, bool clip, double max_norm, double eps, float* norm,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!g || !(norm_type == 1.0 || norm_type == 2.0 || norm_type == HUGE_VAL) || !std::isfinite(scale) ||
      (clip && (!(max_norm >= 0.0) || !(eps >= 0.0) || !std::isfinite(eps))))
    return HBMC_ERR_INVALID_ARG;
  GradArgs a = {};
  a.sums = grad_sums(g->pieces, g->written);
  const uint64_t bytes = workspace_of(g);
  if (workspace_bytes < bytes) return HBMC_ERR_INVALID_ARG;
  Ranges r;
  r.write(norm, 4, 4);
  r.write(workspace, bytes, 16);
  if (!r.ok() || !apart(g, norm, 4) || (bytes > 0 && !apart(g, workspace, bytes))) return HBMC_ERR_INVALID_ARG;
  int device = -1;
  if (hipGetDevice(&device) != hipSuccess) return HBMC_ERR_HIP;
  if (device != g->device) return HBMC_ERR_INVALID_ARG;
  a.pieces = g->piece;
  a.others = g->others;
  a.n = g->pieces;
  a.norm = norm_type == 2.0 ? 2 : norm_type == 1.0 ? 1 : 0;
  a.clip = clip;
  a.read = g->read;
  a.written = g->written;
  a.scale = scale;
  a.max_norm = max_norm;
  a.eps = eps;
  a.partial = static_cast<double*>(workspace);
  a.norm_out = norm;
  return hip(launch_grad(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

hbmc_status_t hbmc_gradients_create(hbmc_comm_t comm, size_t n, const hbmc_gradient_t tensors[], hbmc_gradients_t* out) {
  if (!out) return HBMC_ERR_INVALID_ARG;
  *out = nullptr;
  return no_throw([&]() -> hbmc_status_t {
    std::unique_ptr<hbmc_gradients> g(new hbmc_gradients);
    const hbmc_status_t st = create(comm, n, tensors, g.get());
    if (st == HBMC_OK) *out = g.release();
    return st;
  });
}

hbmc_status_t hbmc_gradients_destroy(hbmc_gradients_t g) {
  if (!g) return HBMC_ERR_INVALID_ARG;
  delete g;
  return HBMC_OK;
}

hbmc_status_t hbmc_gradients_workspace(hbmc_gradients_t g, size_t* bytes) {
  if (!g || !bytes) return HBMC_ERR_INVALID_ARG;
  *bytes = workspace_of(g);
  return HBMC_OK;
}

hbmc_status_t hbmc_gradients_norm(hbmc_gradients_t g, double norm_type, double scale, float* norm, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return no_throw([&] { return run(g, norm_type, scale, false, 0.0, 0.0, norm, workspace, workspace_bytes, stream); });
}

hbmc_status_t hbmc_gradients_clip(hbmc_gradients_t g, double norm_type, double scale, double max_norm, double eps, float* norm,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  return no_throw([&] { return run(g, norm_type, scale, true, max_norm, eps, norm, workspace, workspace_bytes, stream); });
}

}  // extern "C"
