// api_serve.cpp -- the C ABI of generation with states (include/flash_mca.h): linear
// attention with a decay for each head, beam search's selection, the reordering of
// states.  Argument checks; every one runs before anything is queued, and nothing
// is allocated here.
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
  uint64_t n;
};
bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}
bool outputs_clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span &o : outs) {
    for (const Span &i : ins)
      if (overlap(o, i)) return true;
    for (const Span &o2 : outs)
      if (&o2 != &o && overlap(o, o2)) return true;
  }
  return false;
}
bool aligned(std::initializer_list<const void *> ptrs, uintptr_t to) {
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % to) return false;
  return true;
}
fmca_status done(int rc) { return rc == 0 ? FMCA_OK : FMCA_ERR_CUDA; }
bool known(fmca_dtype t) { return t == FMCA_F32 || t == FMCA_BF16; }

static_assert(FMCA_BEAM_MAX == kBeamMax, "the header's limit is the kernels'");

// Every offset of an operand fits 62 bits: a size or stride beyond 2^40 is refused,
// and so is an operand that would span 2^60 bytes.
constexpr int64_t kMost = (int64_t)1 << 40, kSpan = (int64_t)1 << 60;

// Bytes that an operand spans from its first element, or -1.
int64_t span(const int64_t *stride, int B, int T, int heads, int d, int el) {
  const int n[3] = {B, T, heads};
  double most = d;
  int64_t last = d;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (stride[i] < 0 || stride[i] > kMost) return -1;
    most += (double)(n[i] - 1) * (double)stride[i];
    if (most * el > (double)kSpan) return -1;
    last += (int64_t)(n[i] - 1) * stride[i];
  }
  return last * el;
}

struct Spans {
  int64_t q, k, v;
};
fmca_status decay_sizes(const fmca_decay_shape *s, fmca_dtype dtype, Spans *sp) {
  if (!s || !known(dtype)) return FMCA_ERR_INVALID_ARG;
  if (s->B <= 0 || s->T <= 0 || s->H <= 0 || s->dk <= 0 || s->dv <= 0 || s->Hq <= 0 ||
      s->Hk <= 0 || s->Hv <= 0)
    return FMCA_ERR_INVALID_ARG;
  if (s->H % s->Hq || s->H % s->Hk || s->H % s->Hv) return FMCA_ERR_SHAPE;
  if (s->dk > kDecayMaxK) return FMCA_ERR_UNSUPPORTED;
  const int el = dtype == FMCA_BF16 ? 2 : 4;
  // the grid's blocks, whichever kernel and cut: at most two units an SM more than
  // heads and tiles of 32 columns; the state and the outputs in bytes
  const double heads = (double)s->B * s->H;
  if (heads * ((s->dv + 31) / 32) > 1e9 || heads * s->dk * s->dv * 4.0 > (double)kMost ||
      heads * s->T * s->dv * 4.0 > (double)kSpan || s->T > 0x7FFFFFFF - 65536)
    return FMCA_ERR_UNSUPPORTED;
  sp->q = span(s->q_stride, s->B, s->T, s->Hq, s->dk, el);
  sp->k = span(s->k_stride, s->B, s->T, s->Hk, s->dk, el);
  sp->v = span(s->v_stride, s->B, s->T, s->Hv, s->dv, el);
  return sp->q < 0 || sp->k < 0 || sp->v < 0 ? FMCA_ERR_SHAPE : FMCA_OK;
}

DecayArgs decay_args(const void *q, const void *k, const void *v, const float *log_decay,
                     const int32_t *lengths, const float *state_in, void *o, float *state_out,
                     const fmca_decay_shape *s, float scale, fmca_dtype dtype) {
  DecayArgs a{};
  a.q = q, a.k = k, a.v = v;
  a.log_decay = log_decay, a.lengths = lengths;
  a.state_in = state_in, a.o = o, a.state_out = state_out;
  a.B = s->B, a.T = s->T, a.H = s->H;
  a.Hq = s->Hq, a.Hk = s->Hk, a.Hv = s->Hv, a.dk = s->dk, a.dv = s->dv;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = s->q_stride[i];
    a.ks[i] = s->k_stride[i];
    a.vs[i] = s->v_stride[i];
  }
  // the stride of a dimension of one is nobody's
  if (s->B == 1) a.qs[0] = a.ks[0] = a.vs[0] = 0;
  if (s->T == 1) a.qs[1] = a.ks[1] = a.vs[1] = 0;
  if (s->Hq == 1) a.qs[2] = 0;
  if (s->Hk == 1) a.ks[2] = 0;
  if (s->Hv == 1) a.vs[2] = 0;
  a.scale = scale;
  a.bf16 = dtype == FMCA_BF16 ? 1 : 0;
  return a;
}

fmca_status decay_pointers(const DecayArgs &a, const void *state) {
  const uintptr_t el = a.bf16 ? 2 : 4;
  if (!a.q || !a.k || !a.v || !a.log_decay || !a.o) return FMCA_ERR_INVALID_ARG;
  if (!aligned({a.q, a.k, a.v, a.o}, el) || !aligned({a.log_decay, a.lengths}, 4))
    return FMCA_ERR_ALIGN;
  return aligned({a.state_in, a.state_out, state}, a.dv % 4 ? 4 : 16) ? FMCA_OK : FMCA_ERR_ALIGN;
}

// Of either kernel: which one runs goes by the operands' addresses too.
size_t decay_bytes(const DecayArgs &a) {
  const size_t s = decay_bytes_simt(a.B, a.T, a.H, a.dk, a.dv);
  const size_t t = a.bf16 && a.dk <= 128 ? decay_bytes_tc(a.B, a.T, a.H, a.dv) : 0;
  return s > t ? s : t;
}

// Whether one of the rows of a piece shares a byte with `n` bytes at p that come again every
// `again` bytes (0: once).  Rows that are as far apart take the same places of every row, so
// that column ranges of one buffer do not clash though the ranges of their addresses do.
bool clash(const fmca_beam_piece &a, int64_t rows, const void *p, int64_t n, int64_t again) {
  const Span all{a.base, (uint64_t)(rows - 1) * a.row + a.bytes};
  if (!overlap(all, Span{p, (uint64_t)(again > 0 ? (rows - 1) * again : 0) + n})) return false;
  if (again > 0 && again != a.row) return true;
  const intptr_t gap = reinterpret_cast<intptr_t>(p) - reinterpret_cast<intptr_t>(a.base);
  const int64_t at = (gap % a.row + a.row) % a.row;
  return at < a.bytes || at + n > a.row;
}
fmca_status pieces_check(const fmca_beam_piece *p, int n, const int64_t *parent, int B, int K) {
  if (!p || n <= 0 || !parent || B <= 0 || K <= 0) return FMCA_ERR_INVALID_ARG;
  if (K > kBeamMax) return FMCA_ERR_UNSUPPORTED;
  if (!aligned({parent}, 8)) return FMCA_ERR_ALIGN;
  const int64_t rows = (int64_t)B * K;
  for (int i = 0; i < n; ++i) {
    if (p[i].bytes < 0 || p[i].row < p[i].bytes || p[i].row > kMost) return FMCA_ERR_SHAPE;
    if (p[i].bytes == 0) continue;
    if (!p[i].base) return FMCA_ERR_INVALID_ARG;
    if ((double)rows * (double)p[i].row > (double)kSpan ||
        (double)B * ((double)p[i].bytes + 256) / 256 > 2e9)
      return FMCA_ERR_UNSUPPORTED;
    if (clash(p[i], rows, parent, 8 * rows, 0)) return FMCA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (p[j].bytes > 0 && clash(p[i], rows, p[j].base, p[j].bytes, p[j].row))
        return FMCA_ERR_INVALID_ARG;
  }
  return FMCA_OK;
}

// Launches of up to kBeamPieces pieces each.
fmca_status reorder(const fmca_beam_piece *p, int n, const int64_t *parent, int B, int K,
                    fmca_stream_t stream) {
  for (int i = 0; i < n; i += kBeamPieces) {
    BeamPiece q[kBeamPieces];
    const int m = n - i < kBeamPieces ? n - i : kBeamPieces;
    for (int j = 0; j < m; ++j) q[j] = BeamPiece{p[i + j].base, p[i + j].row, p[i + j].bytes, 0};
    const int rc =
        launch_beam_reorder(q, m, parent, B, K, reinterpret_cast<cudaStream_t>(stream));
    if (rc != 0) return FMCA_ERR_CUDA;
  }
  return FMCA_OK;
}

}  // namespace

extern "C" {

size_t flash_mca_decay_workspace_bytes(const fmca_decay_shape *shape, fmca_dtype dtype) {
  Spans sp;
  if (decay_sizes(shape, dtype, &sp) != FMCA_OK) return (size_t)-1;
  return decay_bytes(decay_args(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                nullptr, shape, 1.0f, dtype));
}

fmca_status flash_mca_decay_attention(const void *q, const void *k, const void *v,
                                      const float *log_decay, const int32_t *lengths,
                                      const float *state_in, void *o, float *state_out,
                                      const fmca_decay_shape *shape, float scale,
                                      fmca_dtype dtype, void *workspace, size_t workspace_bytes_,
                                      fmca_stream_t stream) {
  Spans sp;
  fmca_status st = decay_sizes(shape, dtype, &sp);
  if (st != FMCA_OK) return st;
  if (!std::isfinite(scale)) return FMCA_ERR_INVALID_ARG;
  const DecayArgs a = decay_args(q, k, v, log_decay, lengths, state_in, o, state_out, shape, scale,
                                 dtype);
  st = decay_pointers(a, nullptr);
  if (st != FMCA_OK) return st;
  const size_t need = decay_bytes(a);
  if (need > 0) {
    if (!workspace || workspace_bytes_ < need) return FMCA_ERR_WORKSPACE;
    if (!aligned({workspace}, 256)) return FMCA_ERR_ALIGN;
  }
  const uint64_t heads = (uint64_t)a.B * a.H, states = 4 * heads * a.dk * a.dv;
  const Span ws{need > 0 ? workspace : nullptr, workspace_bytes_};
  const Span out{o, heads * a.T * a.dv * (a.bf16 ? 2 : 4)}, so{state_out, states};
  const Span si{state_in == state_out ? nullptr : state_in, states};
  const Span lens{lengths, 4 * (uint64_t)a.B}, rates{log_decay, 4 * (uint64_t)a.H};
  const Span sq{q, (uint64_t)sp.q}, sk{k, (uint64_t)sp.k}, sv{v, (uint64_t)sp.v};
  if (outputs_clash({out, so, ws}, {sq, sk, sv, rates, lens, si}) ||
      overlap(out, Span{state_in, states}) || overlap(ws, Span{state_in, states}))
    return FMCA_ERR_INVALID_ARG;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return done(decay_tc(a) ? launch_tc_decay(a, workspace, cs)
                          : launch_decay_simt(a, workspace, cs));
}

fmca_status flash_mca_decay_step(const void *q, const void *k, const void *v,
                                 const float *log_decay, float *state, void *o,
                                 const fmca_decay_shape *shape, float scale, fmca_dtype dtype,
                                 fmca_stream_t stream) {
  Spans sp;
  fmca_status st = decay_sizes(shape, dtype, &sp);
  if (st != FMCA_OK) return st;
  if (shape->T != 1) return FMCA_ERR_SHAPE;
  if (!std::isfinite(scale) || !state) return FMCA_ERR_INVALID_ARG;
  const DecayArgs a = decay_args(q, k, v, log_decay, nullptr, nullptr, o, nullptr, shape, scale,
                                 dtype);
  st = decay_pointers(a, state);
  if (st != FMCA_OK) return st;
  const uint64_t heads = (uint64_t)a.B * a.H;
  if (outputs_clash({{o, heads * a.dv * (a.bf16 ? 2 : 4)}, {state, 4 * heads * a.dk * a.dv}},
                    {{q, (uint64_t)sp.q}, {k, (uint64_t)sp.k}, {v, (uint64_t)sp.v},
                     {log_decay, 4 * (uint64_t)a.H}}))
    return FMCA_ERR_INVALID_ARG;
  return done(launch_decay_step(a, state, reinterpret_cast<cudaStream_t>(stream)));
}

fmca_status flash_mca_beam_select(const void *logits, int64_t row, const float *scores,
                                  const uint8_t *finished, float *score, int64_t *parent,
                                  int64_t *token, int B, int K, int V, int n, int pad,
                                  fmca_dtype dtype, fmca_stream_t stream) {
  if (B <= 0 || K <= 0 || V <= 0 || n <= 0 || !known(dtype)) return FMCA_ERR_INVALID_ARG;
  if (!logits || !scores || !score || !parent || !token || pad < 0 || pad >= V)
    return FMCA_ERR_INVALID_ARG;
  if (K > kBeamMax || n > kBeamMax) return FMCA_ERR_UNSUPPORTED;
  const uintptr_t el = dtype == FMCA_BF16 ? 2 : 4;
  const uint64_t rows = (uint64_t)B * K, outs = (uint64_t)B * n;
  if (rows > 1 && (row < V || row > kMost)) return FMCA_ERR_SHAPE;
  if (rows == 1) row = 0;
  if ((double)rows * (double)row * (double)el > (double)kSpan ||
      (int64_t)B * kBeamCluster > 0x7FFFFFFF)
    return FMCA_ERR_UNSUPPORTED;
  if (!aligned({logits}, el) || !aligned({scores, score}, 4) || !aligned({parent, token}, 8))
    return FMCA_ERR_ALIGN;
  if (outputs_clash({{score, 4 * outs}, {parent, 8 * outs}, {token, 8 * outs}},
                    {{logits, el * ((rows - 1) * (uint64_t)row + V)}, {scores, 4 * rows},
                     {finished, rows}}))
    return FMCA_ERR_INVALID_ARG;
  return done(launch_beam_select(logits, row, scores, finished, score, parent, token, B, K, V, n,
                                 pad, dtype == FMCA_BF16 ? 1 : 0,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

fmca_status flash_mca_beam_reorder(const fmca_beam_piece *pieces, int n_pieces,
                                   const int64_t *parent, int B, int K, fmca_stream_t stream) {
  const fmca_status st = pieces_check(pieces, n_pieces, parent, B, K);
  return st != FMCA_OK ? st : reorder(pieces, n_pieces, parent, B, K, stream);
}

fmca_status flash_mca_decode_reorder(void *state, size_t state_bytes, const int64_t *parent,
                                     int B, int K, int s, int e, int C, int t, fmca_dtype dtype,
                                     fmca_stream_t stream) {
  if (B <= 0 || K <= 0 || t < 0 || !known(dtype)) return FMCA_ERR_INVALID_ARG;
  if ((int64_t)B * K > 0x7FFFFFFF) return FMCA_ERR_UNSUPPORTED;
  const size_t need = flash_mca_decode_state_bytes(B * K, s, e, C, dtype);
  if (need == 0) return FMCA_ERR_INVALID_ARG;
  if (!state || state_bytes < need) return FMCA_ERR_WORKSPACE;
  if (!aligned({state}, 256)) return FMCA_ERR_ALIGN;
  const int64_t el = dtype == FMCA_BF16 ? 2 : 4, se = (int64_t)s * e, i = t % C;
  const DecodeStateLayout L = decode_state_layout(B * K, s, e, C, (size_t)el);
  char *p = static_cast<char *>(state);
  // the rows of the chunk that holds position t, so far (none at its first one: the
  // chunk before it is in the sums)
  const fmca_beam_piece pieces[4] = {{p + L.P, 4 * se, 4 * se},
                                     {p + L.Pb, 2 * se, el == 2 ? 2 * se : 0},
                                     {p + L.Zc, el * C * s, el * i * s},
                                     {p + L.Vc, el * C * e, el * i * e}};
  const fmca_status st = pieces_check(pieces, 4, parent, B, K);
  return st != FMCA_OK ? st : reorder(pieces, 4, parent, B, K, stream);
}

}  // extern "C"
