// api_train.cpp -- the C ABI of the training operators around the attention
// core (include/flash_mca.h): argument checks and workspace sizing.  Every
// check runs before anything is queued; no allocation happens here.
#include "flash_mca.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "launch.h"

using namespace fmca;

namespace {

struct Span {
  const void *p;
  size_t n;
};
bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}
// outputs must not overlap the inputs or each other
bool outputs_clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span &o : outs) {
    for (const Span &i : ins)
      if (overlap(o, i)) return true;
    for (const Span &o2 : outs)
      if (&o2 != &o && overlap(o, o2)) return true;
  }
  return false;
}
// NULL counts as aligned
bool aligned(std::initializer_list<const void *> ptrs, uintptr_t to) {
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % to) return false;
  return true;
}
fmca_status done(int rc) { return rc == 0 ? FMCA_OK : FMCA_ERR_CUDA; }

fmca_status norm_sizes(int M, int d) {
  if (M <= 0 || d <= 0) return FMCA_ERR_INVALID_ARG;
  if (d > kNormMaxD) return FMCA_ERR_UNSUPPORTED;
  return FMCA_OK;
}

constexpr int64_t kLimit = (int64_t)1 << 31;

fmca_status project_sizes(int M, int d, int e, int s) {
  if (M <= 0 || d <= 0 || e <= 0 || s <= 0) return FMCA_ERR_INVALID_ARG;
  if (d % 8 || e % 64 || s % 64) return FMCA_ERR_UNSUPPORTED;
  const int64_t N = 2 * (int64_t)e + s;
  if (M * N >= kLimit || (int64_t)M * d >= kLimit || N * d >= kLimit) return FMCA_ERR_UNSUPPORTED;
  return FMCA_OK;
}
fmca_status output_sizes(int M, int e, int d) {
  if (M <= 0 || d <= 0 || e <= 0) return FMCA_ERR_INVALID_ARG;
  if (e % 8 || d % 64) return FMCA_ERR_UNSUPPORTED;
  if ((int64_t)M * (e > d ? e : d) >= kLimit || (int64_t)d * e >= kLimit)
    return FMCA_ERR_UNSUPPORTED;
  return FMCA_OK;
}
// The logits' depth is not cut: 2^24 features are 2^18 k steps of a tile, 0.2 s at
// a CTA's share of the memory's rate, of the second that a wait may take.
constexpr int kVocabMaxD = 1 << 24;
fmca_status vocab_sizes(int M, int V, int d) {
  if (M <= 0 || V <= 0 || d <= 0) return FMCA_ERR_INVALID_ARG;
  if (d % 8 || d > kVocabMaxD || (int64_t)M * d >= kLimit || (int64_t)V * d >= kLimit)
    return FMCA_ERR_UNSUPPORTED;
  return FMCA_OK;
}
fmca_status check_workspace(const void *workspace, size_t have, size_t need) {
  if (!workspace || have < need) return FMCA_ERR_WORKSPACE;
  return aligned({workspace}, 256) ? FMCA_OK : FMCA_ERR_ALIGN;
}

}  // namespace

extern "C" {

fmca_status flash_mca_layer_norm(const void *x, const void *res, const float *weight,
                                 const float *bias, void *h, void *y, float *mean, float *rstd,
                                 int M, int d, float eps, fmca_dtype dtype,
                                 fmca_stream_t stream) {
  const fmca_status st = norm_sizes(M, d);
  if (st != FMCA_OK) return st;
  if (dtype != FMCA_F32 && dtype != FMCA_BF16) return FMCA_ERR_INVALID_ARG;
  if (!x || !weight || !bias || !y || (res && !h)) return FMCA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.0f) return FMCA_ERR_INVALID_ARG;
  if (!aligned({x, res, weight, bias, y}, 16) || !aligned({mean, rstd}, 4)) return FMCA_ERR_ALIGN;
  const size_t rows = (size_t)M * d * (dtype == FMCA_BF16 ? 2 : 4);
  const size_t wb = sizeof(float) * (size_t)d, sb = sizeof(float) * (size_t)M;
  void *const hh = res ? h : nullptr;  // without a residual branch h is not touched
  if (!aligned({hh}, 16)) return FMCA_ERR_ALIGN;
  if (outputs_clash({{y, rows}, {mean, sb}, {rstd, sb}},
                    {{x, rows}, {res, rows}, {weight, wb}, {bias, wb}, {hh, rows}}))
    return FMCA_ERR_INVALID_ARG;
  // h: x or res itself (every thread has read its elements before it writes
  // them), or apart from every input
  if (hh && ((hh != x && overlap({hh, rows}, {x, rows})) ||
             (hh != res && overlap({hh, rows}, {res, rows})) ||
             overlap({hh, rows}, {weight, wb}) || overlap({hh, rows}, {bias, wb})))
    return FMCA_ERR_INVALID_ARG;
  return done(launch_layer_norm(x, res, weight, bias, hh, y, mean, rstd, M, d, eps,
                                dtype == FMCA_BF16 ? 1 : 0,
                                reinterpret_cast<cudaStream_t>(stream)));
}

size_t flash_mca_layer_norm_backward_workspace_bytes(int M, int d) {
  return norm_sizes(M, d) == FMCA_OK ? norm_backward_bytes(M, d) : 0;
}

fmca_status flash_mca_layer_norm_backward(const void *dy, const void *h, const float *weight,
                                          const float *mean, const float *rstd, const void *dh,
                                          void *dx, float *dweight, float *dbias, int M, int d,
                                          fmca_dtype dtype, void *workspace,
                                          size_t workspace_bytes_, fmca_stream_t stream) {
  const fmca_status st = norm_sizes(M, d);
  if (st != FMCA_OK) return st;
  if (dtype != FMCA_F32 && dtype != FMCA_BF16) return FMCA_ERR_INVALID_ARG;
  if (!dy || !h || !weight || !mean || !rstd || !dx || !dweight || !dbias)
    return FMCA_ERR_INVALID_ARG;
  if (!aligned({dy, h, weight, dh, dx, dweight, dbias}, 16) || !aligned({mean, rstd}, 4))
    return FMCA_ERR_ALIGN;
  if (!workspace || workspace_bytes_ < norm_backward_bytes(M, d)) return FMCA_ERR_WORKSPACE;
  if (!aligned({workspace}, 256)) return FMCA_ERR_ALIGN;
  const size_t rows = (size_t)M * d * (dtype == FMCA_BF16 ? 2 : 4);
  const size_t wb = sizeof(float) * (size_t)d, sb = sizeof(float) * (size_t)M;
  if (outputs_clash({{dx, rows}, {dweight, wb}, {dbias, wb}, {workspace, workspace_bytes_}},
                    {{dy, rows}, {h, rows}, {weight, wb}, {mean, sb}, {rstd, sb}, {dh, rows}}))
    return FMCA_ERR_INVALID_ARG;
  return done(launch_layer_norm_backward(dy, h, weight, mean, rstd, dh, dx, dweight, dbias, M, d,
                                         dtype == FMCA_BF16 ? 1 : 0, workspace,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

size_t flash_mca_gau_project_backward_workspace_bytes(int M, int d, int e, int s) {
  return project_sizes(M, d, e, s) == FMCA_OK ? project_grad_layout(M, 2 * e + s).total : 0;
}

fmca_status flash_mca_gau_project_backward(const void *X, const void *Wt, const void *dU,
                                           const void *dV, const void *dZ, void *dX, void *dWt,
                                           int M, int d, int e, int s, void *workspace,
                                           size_t workspace_bytes_, fmca_stream_t stream) {
  fmca_status st = project_sizes(M, d, e, s);
  if (st != FMCA_OK) return st;
  if (!X || !Wt || !dU || !dV || !dZ || !dX || !dWt) return FMCA_ERR_INVALID_ARG;
  if (!aligned({X, Wt, dU, dV, dZ, dX, dWt}, 16)) return FMCA_ERR_ALIGN;
  st = check_workspace(workspace, workspace_bytes_, project_grad_layout(M, 2 * e + s).total);
  if (st != FMCA_OK) return st;
  const size_t xb = 2 * (size_t)M * d, wb = 2 * (size_t)(2 * (int64_t)e + s) * d;
  const size_t eb = 2 * (size_t)M * e, zb = 2 * (size_t)M * s;
  if (outputs_clash({{dX, xb}, {dWt, wb}, {workspace, workspace_bytes_}},
                    {{X, xb}, {Wt, wb}, {dU, eb}, {dV, eb}, {dZ, zb}}))
    return FMCA_ERR_INVALID_ARG;
  return done(launch_gau_project_backward(X, Wt, dU, dV, dZ, dX, dWt, M, d, e, s, workspace,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

size_t flash_mca_gau_output_backward_workspace_bytes(int M, int e, int d) {
  return output_sizes(M, e, d) == FMCA_OK ? output_grad_layout().total : 0;
}

fmca_status flash_mca_gau_output_backward(const void *Y, const void *Wo_t, const void *dOut,
                                          void *dY, void *dWo_t, int M, int e, int d,
                                          void *workspace, size_t workspace_bytes_,
                                          fmca_stream_t stream) {
  fmca_status st = output_sizes(M, e, d);
  if (st != FMCA_OK) return st;
  if (!Y || !Wo_t || !dOut || !dY || !dWo_t) return FMCA_ERR_INVALID_ARG;
  if (!aligned({Y, Wo_t, dOut, dY, dWo_t}, 16)) return FMCA_ERR_ALIGN;
  st = check_workspace(workspace, workspace_bytes_, output_grad_layout().total);
  if (st != FMCA_OK) return st;
  const size_t yb = 2 * (size_t)M * e, wb = 2 * (size_t)d * e, ob = 2 * (size_t)M * d;
  if (outputs_clash({{dY, yb}, {dWo_t, wb}, {workspace, workspace_bytes_}},
                    {{Y, yb}, {Wo_t, wb}, {dOut, ob}}))
    return FMCA_ERR_INVALID_ARG;
  return done(launch_gau_output_backward(Y, Wo_t, dOut, dY, dWo_t, M, e, d, workspace,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

size_t flash_mca_vocab_loss_workspace_bytes(int M, int V, int d) {
  return vocab_sizes(M, V, d) == FMCA_OK ? vocab_loss_layout(M, V, d).total : 0;
}

fmca_status flash_mca_vocab_loss(const void *X, const void *W, const int64_t *target, float *loss,
                                 float *lse, int M, int V, int d, void *workspace,
                                 size_t workspace_bytes_, fmca_stream_t stream) {
  fmca_status st = vocab_sizes(M, V, d);
  if (st != FMCA_OK) return st;
  if (!X || !W || !target || !loss || !lse) return FMCA_ERR_INVALID_ARG;
  if (!aligned({X, W}, 16) || !aligned({target}, 8) || !aligned({loss, lse}, 4))
    return FMCA_ERR_ALIGN;
  st = check_workspace(workspace, workspace_bytes_, vocab_loss_layout(M, V, d).total);
  if (st != FMCA_OK) return st;
  const size_t xb = 2 * (size_t)M * d, wb = 2 * (size_t)V * d, rb = 4 * (size_t)M;
  if (outputs_clash({{loss, rb}, {lse, rb}, {workspace, workspace_bytes_}},
                    {{X, xb}, {W, wb}, {target, 2 * rb}}))
    return FMCA_ERR_INVALID_ARG;
  return done(launch_vocab_loss(X, W, target, loss, lse, M, V, d, workspace,
                                reinterpret_cast<cudaStream_t>(stream)));
}

size_t flash_mca_vocab_loss_backward_workspace_bytes(int M, int V, int d) {
  return vocab_sizes(M, V, d) == FMCA_OK ? vocab_grad_layout(M, V, d).total : 0;
}

fmca_status flash_mca_vocab_loss_backward(const void *X, const void *W, const int64_t *target,
                                          const float *lse, const float *dloss, void *dX, void *dW,
                                          int M, int V, int d, void *workspace,
                                          size_t workspace_bytes_, fmca_stream_t stream) {
  fmca_status st = vocab_sizes(M, V, d);
  if (st != FMCA_OK) return st;
  if (!X || !W || !target || !lse || !dloss || !dX || !dW) return FMCA_ERR_INVALID_ARG;
  if (!aligned({X, W, dX, dW}, 16) || !aligned({target}, 8) || !aligned({lse, dloss}, 4))
    return FMCA_ERR_ALIGN;
  st = check_workspace(workspace, workspace_bytes_, vocab_grad_layout(M, V, d).total);
  if (st != FMCA_OK) return st;
  const size_t xb = 2 * (size_t)M * d, wb = 2 * (size_t)V * d, rb = 4 * (size_t)M;
  if (outputs_clash({{dX, xb}, {dW, wb}, {workspace, workspace_bytes_}},
                    {{X, xb}, {W, wb}, {target, 2 * rb}, {lse, rb}, {dloss, rb}}))
    return FMCA_ERR_INVALID_ARG;
  return done(launch_vocab_loss_backward(X, W, target, lse, dloss, dX, dW, M, V, d, workspace,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
