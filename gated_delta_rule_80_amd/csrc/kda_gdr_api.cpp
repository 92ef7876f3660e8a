// Host side of the gated delta rule with one decay per head and of the page
// operations: argument validation (host-only, no HIP calls), workspace sizing and
// the launch sequence on the caller's stream.  See include/kda.h.
#include "kda.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "kda_gdr.h"
#include "kda_host.h"
#include "kda_launch.h"

namespace {

using namespace kda;

constexpr uint32_t kGdrFlags = KDA_FLAG_L2NORM_QK | KDA_FLAG_BETA_LOGITS;

bool gdr_dim(int D) { return D == 32 || D == 64 || D == 128; }

// bytes of `rows` rows of `row` elements, `stride` elements apart (0: packed)
bool rows_bytes(size_t& out, size_t rows, size_t row, int64_t stride, size_t es) {
  if (rows == 0) {
    out = 0;
    return true;
  }
  const size_t st = stride > 0 ? (size_t)stride : row;
  size_t body;
  if (!mul_ok(body, {rows - 1, st, es}) || row > (size_t(1) << 40)) return false;
  out = body + row * es;
  return true;
}

// a stride is 0, or holds the row and keeps its 16-byte pieces aligned; the kernels
// address the rows of a chunk by 32-bit offsets
bool stride_ok(int64_t stride, size_t row, size_t es) {
  return row <= (size_t(1) << 23) &&
         (stride == 0 || (stride >= (int64_t)row && (size_t)stride * es % 16 == 0 && stride <= (int64_t(1) << 23)));
}

constexpr size_t kGdrMaxGroups = (size_t(1) << 23) - 1;

struct GdrSizes {
  size_t q, k, v, o, gates, state, cu;  // bytes
  int NS, NT;
};

bool gdr_packed(const kda_gdr_args* a) { return a->cu_seqlens != nullptr; }

kda_status gdr_sizes(const kda_gdr_args* a, GdrSizes& s) {
  const size_t es = esize(a->io);
  const int C = gdr_chunk(a->io == KDA_FP32);
  s.NS = gdr_packed(a) ? a->n_seqs : a->B;
  size_t tok;
  if (!mul_ok(tok, {(size_t)a->B, (size_t)a->T})) return KDA_ERR_SHAPE;
  const size_t rk = (size_t)a->Hk * a->Dk, rv = (size_t)a->Hv * a->Dv;
  if (!rows_bytes(s.q, tok, rk, a->q_stride, es) || !rows_bytes(s.k, tok, rk, a->k_stride, es) ||
      !rows_bytes(s.v, tok, rv, a->v_stride, es) || !mul_ok(s.o, {tok, rv, es}) ||
      !mul_ok(s.gates, {tok, (size_t)a->Hv, es}) ||
      !mul_ok(s.state, {(size_t)s.NS, (size_t)a->Hv, (size_t)a->Dk, (size_t)a->Dv, 4}))
    return KDA_ERR_SHAPE;
  s.cu = gdr_packed(a) ? ((size_t)a->n_seqs + 1) * 4 : 0;
  const long nt = ((long)a->T + C - 1) / C;
  // packed: every sequence wastes at most one partly filled chunk
  const long slots = gdr_packed(a) && a->T > 0 ? nt + a->n_seqs : nt;
  if (slots > 0x7fffffffL) return KDA_ERR_SHAPE;
  s.NT = (int)slots;
  // a launch holds less than 2^32 threads, a workgroup up to 512 of them: one per
  // chunk and head, and up to two per sequence and head (rounded up, gdr_walk_grid)
  size_t wgs;
  if (!mul_ok(wgs, {(size_t)a->B, (size_t)a->Hv, (size_t)(s.NT > 0 ? s.NT : 1)}) || wgs > kGdrMaxGroups ||
      !mul_ok(wgs, {(size_t)s.NS + 8, (size_t)a->Hv, 2}) || wgs > kGdrMaxGroups)
    return KDA_ERR_SHAPE;
  return KDA_OK;
}

// everything but the outputs o and S_T
kda_status gdr_validate_inputs(const kda_gdr_args* a, GdrSizes& s) {
  if (a->io != KDA_BF16 && a->io != KDA_FP32) return KDA_ERR_DTYPE;
  if (a->B < 1 || a->T < 0 || a->Hk < 1 || a->Hv < 1 || a->Dk < 1 || a->Dv < 1) return KDA_ERR_SHAPE;
  if (a->Hv % a->Hk != 0) return KDA_ERR_SHAPE;
  if (!gdr_dim(a->Dk) || !gdr_dim(a->Dv)) return KDA_ERR_UNSUPPORTED;
  if ((a->flags & ~kGdrFlags) != 0) return KDA_ERR_VALUE;
  if (!std::isfinite(a->l2_eps) || a->l2_eps < 0.f || !std::isfinite(a->scale)) return KDA_ERR_VALUE;
  if (gdr_packed(a) ? (a->B != 1 || a->n_seqs < 1) : a->n_seqs != 0) return KDA_ERR_SHAPE;
  const size_t es = esize(a->io);
  if (!stride_ok(a->q_stride, (size_t)a->Hk * a->Dk, es) || !stride_ok(a->k_stride, (size_t)a->Hk * a->Dk, es) ||
      !stride_ok(a->v_stride, (size_t)a->Hv * a->Dv, es))
    return KDA_ERR_SHAPE;
  if (kda_status e = gdr_sizes(a, s); e != KDA_OK) return e;
  if ((a->A_log == nullptr) != (a->dt_bias == nullptr)) return KDA_ERR_NULL;
  if (a->T > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta)) return KDA_ERR_NULL;
  for (const void* p : std::initializer_list<const void*>{a->q, a->k, a->v, a->g, a->beta, a->S0, a->A_log,
                                                          a->dt_bias, a->cu_seqlens})
    if (p && !aligned16(p)) return KDA_ERR_ALIGN;
  return KDA_OK;
}

// A few address ranges (no allocation: nothing here may throw at a C entry).
struct Spans {
  Span s[24];
  int n = 0;
  Spans(std::initializer_list<Span> xs) {
    for (Span x : xs) add(x);
  }
  void add(Span x) {
    if (n < 24) s[n++] = x;
  }
  const Span* begin() const { return s; }
  const Span* end() const { return s + n; }
};

Spans gdr_inputs(const kda_gdr_args* a, const GdrSizes& s) {
  return {span(a->S0, s.state), span(a->q, s.q), span(a->k, s.k), span(a->v, s.v), span(a->g, s.gates),
          span(a->beta, s.gates), span(a->A_log, (size_t)a->Hv * 4), span(a->dt_bias, (size_t)a->Hv * 4),
          span(a->cu_seqlens, s.cu)};
}

// outputs overlap no input and none another
kda_status disjoint(const Spans& outs, const Spans& ins) {
  for (int i = 0; i < outs.n; ++i) {
    for (const Span& x : ins)
      if (overlaps(outs.s[i], x)) return KDA_ERR_ALIAS;
    for (int j = i + 1; j < outs.n; ++j)
      if (overlaps(outs.s[i], outs.s[j])) return KDA_ERR_ALIAS;
  }
  return KDA_OK;
}

// The workspace: sequence tables, the chunk records, for the backward Y, the two
// checkpoints per chunk and the float32 gradient of the decay, and of a split walk the
// segments' starts, maps and (backward) ends.
struct GdrWork {
  size_t seq, segs, rec, y, ckS, ckdS, dg, starts, maps, ends, bytes;
};
GdrSplit split_of(const kda_gdr_args* a, const GdrSizes& s, bool bwd) {
  if (a->T == 0 || (gdr_packed(a) && bwd)) return {1, s.NT};
  if (gdr_packed(a))
    return gdr_split_packed(a->T, gdr_chunk(a->io == KDA_FP32), a->n_seqs, a->Hv, a->Dv, a->io == KDA_FP32);
  return gdr_split((long)a->B * a->Hv, s.NT, a->Dv, a->io == KDA_FP32, bwd);
}
bool gdr_work(const kda_gdr_args* a, const GdrSizes& s, bool bwd, GdrWork& w) {
  const size_t es = esize(a->io);
  size_t nrec, recs, ck = 0, y = 0, dg = 0;
  if (!mul_ok(nrec, {(size_t)a->B, (size_t)a->Hv, (size_t)s.NT}) ||
      !mul_ok(recs, {nrec, gdr_record(a->io == KDA_FP32, bwd).bytes}))
    return false;
  if (bwd) {
    if (!mul_ok(ck, {nrec, (size_t)a->Dk, (size_t)a->Dv, es})) return false;
    y = s.o;
    dg = a->A_log != nullptr ? s.gates / es * 4 : 0;
  }
  w.seq = 0;
  // the tables of chunks, and of a split walk those of segments
  w.segs = round_up(gdr_packed(a) ? 8 * ((size_t)a->n_seqs + 1) : 0, 256);
  w.rec = w.segs + (gdr_packed(a) && split_of(a, s, bwd).nseg > 1 ? round_up(8 * ((size_t)a->n_seqs + 1), 256) : 0);
  w.y = w.rec + recs;
  w.ckS = round_up(w.y + y, 256);
  w.ckdS = round_up(w.ckS + ck, 256);
  w.dg = round_up(w.ckdS + ck, 256);
  w.starts = w.maps = w.ends = round_up(w.dg + dg, 256);
  w.bytes = w.starts;
  if (const GdrSplit sp = split_of(a, s, bwd); sp.nseg > 1) {
    // about 256 workgroups of segments: these sizes stay small
    const size_t n = (size_t)a->B * a->Hv * sp.nseg * a->Dk * 4;
    w.maps = w.starts + n * a->Dv;
    w.ends = w.maps + n * a->Dk;
    w.bytes = w.ends + (bwd ? n * a->Dv : 0);
  }
  return w.bytes < (size_t(1) << 62);
}

kda_status gdr_check_ws(void* ws, size_t ws_bytes, size_t need, const Spans& others) {
  if (need == 0) return KDA_OK;
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < need)
    return KDA_ERR_WORKSPACE;
  const Span w = span(ws, need);
  for (const Span& x : others)
    if (overlaps(w, x)) return KDA_ERR_ALIAS;
  return KDA_OK;
}

GdrShape gdr_shape(const kda_gdr_args* a, const GdrSizes& s, char* ws, const GdrWork& w) {
  GdrShape g{};
  g.B = a->B; g.T = a->T; g.Hk = a->Hk; g.Hv = a->Hv;
  g.NS = s.NS; g.NT = s.NT;
  g.qs = a->q_stride > 0 ? a->q_stride : (long)a->Hk * a->Dk;
  g.ks = a->k_stride > 0 ? a->k_stride : (long)a->Hk * a->Dk;
  g.vs = a->v_stride > 0 ? a->v_stride : (long)a->Hv * a->Dv;
  if (gdr_packed(a) && a->T > 0) {
    int* bounds = reinterpret_cast<int*>(ws + w.seq);
    g.seqs.bounds = bounds;
    g.seqs.cstart = bounds + a->n_seqs + 1;
    g.seqs.n_seqs = a->n_seqs;
  }
  return g;
}

// sequence tables and chunk records
kda_status gdr_prepare(const kda_gdr_args* a, const GdrShape& g, char* rec, bool bwd, hipStream_t st) {
  if (g.seqs.bounds != nullptr) {
    IndexParams ip{};
    ip.cu_seqlens = a->cu_seqlens;
    ip.bounds = const_cast<int*>(g.seqs.bounds);
    ip.cstart = const_cast<int*>(g.seqs.cstart);
    ip.n_seqs = a->n_seqs;
    ip.T = a->T;
    ip.C = gdr_chunk(a->io == KDA_FP32);
    if (kda_status e = hip_status(launch_seq_index(ip, st)); e != KDA_OK) return e;
  }
  GdrPrepParams p{};
  p.s = g;
  p.q = a->q; p.k = a->k; p.g = a->g; p.beta = a->beta;
  p.A_log = a->A_log; p.dt_bias = a->dt_bias;
  p.beta_logits = (a->flags & KDA_FLAG_BETA_LOGITS) != 0;
  p.l2 = (a->flags & KDA_FLAG_L2NORM_QK) != 0;
  p.eps = a->l2_eps; p.scale = a->scale;
  p.rec = rec;
  return hip_status(launch_gdr_prep(p, a->Dk, a->io == KDA_FP32, bwd, st));
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ prefill
kda_status kda_validate_gdr_prefill(const kda_gdr_args* a) {
  if (a == nullptr) return KDA_ERR_NULL;
  GdrSizes s;
  if (kda_status e = gdr_validate_inputs(a, s); e != KDA_OK) return e;
  if (!a->S_T || (a->T > 0 && !a->o)) return KDA_ERR_NULL;
  if (!aligned16(a->S_T) || (a->o && !aligned16(a->o))) return KDA_ERR_ALIGN;
  const Span st = span(a->S_T, s.state), s0 = span(a->S0, s.state);
  Spans ins = gdr_inputs(a, s);
  const Span o = span(a->o, s.o);
  if (kda_status e = disjoint({o}, ins); e != KDA_OK) return e;
  ins.s[0] = Span{};  // S0: the state may be updated in place
  if (!same_or_disjoint(st, s0)) return KDA_ERR_ALIAS;
  return disjoint({o, st}, ins);
}

size_t kda_gdr_prefill_workspace_bytes(const kda_gdr_args* a) {
  if (kda_validate_gdr_prefill(a) != KDA_OK || a->T == 0) return 0;
  GdrSizes s;
  GdrWork w;
  gdr_sizes(a, s);
  return gdr_work(a, s, false, w) ? w.bytes : 0;
}

kda_status kda_gdr_prefill(const kda_gdr_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (kda_status e = kda_validate_gdr_prefill(a); e != KDA_OK) return e;
  GdrSizes s;
  GdrWork w;
  gdr_sizes(a, s);
  if (!gdr_work(a, s, false, w)) return KDA_ERR_SHAPE;
  Spans all = gdr_inputs(a, s);
  all.add(span(a->o, s.o));
  all.add(span(a->S_T, s.state));
  if (kda_status e = gdr_check_ws(ws, ws_bytes, a->T > 0 ? w.bytes : 0, all); e != KDA_OK) return e;
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* base = static_cast<char*>(ws);
  if (a->T == 0) {
    if (a->S_T == a->S0) return KDA_OK;
    return hip_status(launch_copy_state(a->S0, a->S_T, s.state / 4, st));
  }
  const GdrShape g = gdr_shape(a, s, base, w);
  if (kda_status e = gdr_prepare(a, g, base + w.rec, false, st); e != KDA_OK) return e;
  GdrWalkParams p{};
  p.s = g;
  p.q = a->q; p.k = a->k; p.v = a->v;
  p.rec = base + w.rec;
  p.S0 = a->S0; p.S_T = a->S_T; p.o = a->o;
  const GdrSplit sp = split_of(a, s, false);
  if (gdr_packed(a) && sp.nseg > 1) {
    IndexParams ip{};
    ip.cu_seqlens = a->cu_seqlens;
    ip.bounds = reinterpret_cast<int*>(base + w.segs);
    ip.cstart = ip.bounds + a->n_seqs + 1;
    ip.n_seqs = a->n_seqs;
    ip.T = a->T;
    ip.C = gdr_chunk(a->io == KDA_FP32) * sp.seg_len;
    p.segstart = ip.cstart;
    if (kda_status e = hip_status(launch_seq_index(ip, st)); e != KDA_OK) return e;
  }
  p.nseg = sp.nseg;
  p.seg_len = sp.seg_len;
  p.starts = reinterpret_cast<float*>(base + w.starts);
  p.maps = reinterpret_cast<float*>(base + w.maps);
  return hip_status(launch_gdr_walk(p, a->Dk, a->Dv, a->io == KDA_FP32, st));
}

// ------------------------------------------------------------------ backward
kda_status kda_validate_gdr_backward(const kda_gdr_backward_args* a) {
  if (a == nullptr) return KDA_ERR_NULL;
  const kda_gdr_args* f = &a->fwd;
  GdrSizes s;
  if (kda_status e = gdr_validate_inputs(f, s); e != KDA_OK) return e;
  if (f->T > 0 && (!a->dO || !a->dq || !a->dk || !a->dv || !a->dg || !a->dbeta)) return KDA_ERR_NULL;
  if (f->A_log == nullptr && (a->dA_log || a->ddt_bias)) return KDA_ERR_NULL;
  for (const void* p : std::initializer_list<const void*>{a->dO, a->dS_T, a->dq, a->dk, a->dv, a->dg, a->dbeta,
                                                          a->dS0, a->dA_log, a->ddt_bias})
    if (p && !aligned16(p)) return KDA_ERR_ALIGN;
  const size_t es = esize(f->io);
  size_t xk;
  if (!mul_ok(xk, {(size_t)f->B, (size_t)f->T, (size_t)f->Hk, (size_t)f->Dk, es})) return KDA_ERR_SHAPE;
  GdrWork w;
  if (!gdr_work(f, s, true, w)) return KDA_ERR_SHAPE;
  Spans ins = gdr_inputs(f, s);
  ins.add(span(a->dO, s.o));
  ins.add(span(a->dS_T, s.state));
  return disjoint({span(a->dq, xk), span(a->dk, xk), span(a->dv, s.o), span(a->dg, s.gates),
                   span(a->dbeta, s.gates), span(a->dS0, s.state), span(a->dA_log, (size_t)f->Hv * 4),
                   span(a->ddt_bias, (size_t)f->Hv * 4)},
                  ins);
}

size_t kda_gdr_backward_workspace_bytes(const kda_gdr_backward_args* a) {
  if (kda_validate_gdr_backward(a) != KDA_OK || a->fwd.T == 0) return 0;
  GdrSizes s;
  GdrWork w;
  gdr_sizes(&a->fwd, s);
  return gdr_work(&a->fwd, s, true, w) ? w.bytes : 0;
}

kda_status kda_gdr_prefill_backward(const kda_gdr_backward_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (kda_status e = kda_validate_gdr_backward(a); e != KDA_OK) return e;
  const kda_gdr_args* f = &a->fwd;
  const bool fp32 = f->io == KDA_FP32;
  hipStream_t st = static_cast<hipStream_t>(stream);
  GdrSizes s;
  GdrWork w;
  gdr_sizes(f, s);
  if (!gdr_work(f, s, true, w)) return KDA_ERR_SHAPE;
  size_t xk = 0;
  mul_ok(xk, {(size_t)f->B, (size_t)f->T, (size_t)f->Hk, (size_t)f->Dk, esize(f->io)});
  Spans all = gdr_inputs(f, s);
  for (Span x : {span(a->dO, s.o), span(a->dS_T, s.state), span(a->dq, xk), span(a->dk, xk), span(a->dv, s.o),
                 span(a->dg, s.gates), span(a->dbeta, s.gates), span(a->dS0, s.state),
                 span(a->dA_log, (size_t)f->Hv * 4), span(a->ddt_bias, (size_t)f->Hv * 4)})
    all.add(x);
  if (kda_status e = gdr_check_ws(ws, ws_bytes, f->T > 0 ? w.bytes : 0, all); e != KDA_OK) return e;
  if (f->T == 0) {
    // no tokens: dS0 = dS_T, and nothing flows into the parameters
    if (a->dS0 != nullptr)
      if (kda_status e = hip_status(launch_copy_state(a->dS_T, a->dS0, s.state / 4, st)); e != KDA_OK) return e;
    for (float* x : {a->dA_log, a->ddt_bias})
      if (x != nullptr)
        if (kda_status e = hip_status(launch_copy_state(nullptr, x, (size_t)f->Hv, st)); e != KDA_OK) return e;
    return KDA_OK;
  }
  char* base = static_cast<char*>(ws);
  const GdrShape g = gdr_shape(f, s, base, w);
  if (kda_status e = gdr_prepare(f, g, base + w.rec, true, st); e != KDA_OK) return e;
  GdrWalkParams p{};
  p.s = g;
  p.q = f->q; p.k = f->k; p.v = f->v;
  p.rec = base + w.rec;
  p.S0 = f->S0;
  p.y = base + w.y;
  p.ckpt = base + w.ckS;
  p.bwd = 1;
  const GdrSplit sp = split_of(f, s, true);
  p.nseg = sp.nseg;
  p.seg_len = sp.seg_len;
  p.starts = reinterpret_cast<float*>(base + w.starts);
  p.maps = reinterpret_cast<float*>(base + w.maps);
  GdrReverseParams rv{};
  rv.s = g;
  rv.q = f->q; rv.k = f->k;
  rv.rec = base + w.rec;
  rv.dO = a->dO; rv.dS_T = a->dS_T; rv.dS0 = a->dS0;
  rv.dv = a->dv;
  rv.ckpt = base + w.ckdS;
  rv.nseg = sp.nseg;
  rv.seg_len = sp.seg_len;
  rv.ends = reinterpret_cast<float*>(base + w.ends);
  if (kda_status e = hip_status(launch_gdr_two_walks(rv, p, f->Dk, f->Dv, fp32, st)); e != KDA_OK) return e;
  GdrGradParams d{};
  d.s = g;
  d.q = f->q; d.k = f->k;
  d.rec = base + w.rec;
  d.dO = a->dO; d.dv = a->dv; d.y = base + w.y;
  d.ckS = base + w.ckS; d.ckdS = base + w.ckdS;
  d.dq = a->dq; d.dk = a->dk; d.dg = a->dg; d.dbeta = a->dbeta;
  d.dg32 = reinterpret_cast<float*>(base + w.dg);
  d.l2 = (f->flags & KDA_FLAG_L2NORM_QK) != 0;
  d.scale = f->scale;
  d.g = f->g; d.A_log = f->A_log; d.dt_bias = f->dt_bias;
  d.beta_logits = (f->flags & KDA_FLAG_BETA_LOGITS) != 0;
  if (kda_status e = hip_status(launch_gdr_grad(d, f->Dk, f->Dv, fp32, st)); e != KDA_OK) return e;
  if (a->dA_log != nullptr || a->ddt_bias != nullptr) {
    GdrGateParams q{};
    q.g = f->g; q.A_log = f->A_log; q.dt_bias = f->dt_bias;
    q.dg32 = d.dg32;
    q.dA_log = a->dA_log; q.ddt_bias = a->ddt_bias;
    q.tokens = (long)f->B * f->T;
    q.Hv = f->Hv;
    q.seqs = g.seqs;
    return hip_status(launch_gdr_gate(q, fp32, st));
  }
  return KDA_OK;
}

// ------------------------------------------------------------------ decode
kda_status kda_validate_gdr_decode(const kda_gdr_decode_args* a) {
  if (a == nullptr) return KDA_ERR_NULL;
  if (a->io != KDA_BF16 && a->io != KDA_FP32) return KDA_ERR_DTYPE;
  if (a->N < 0 || a->n_slots < 1 || a->Hk < 1 || a->Hv < 1 || a->Dk < 1 || a->Dv < 1) return KDA_ERR_SHAPE;
  if (a->Hv % a->Hk != 0) return KDA_ERR_SHAPE;
  if (!gdr_dim(a->Dk) || !gdr_dim(a->Dv)) return KDA_ERR_UNSUPPORTED;
  if ((a->flags & ~kGdrFlags) != 0) return KDA_ERR_VALUE;
  if (!std::isfinite(a->l2_eps) || a->l2_eps < 0.f || !std::isfinite(a->scale)) return KDA_ERR_VALUE;
  if (a->slots == nullptr && a->N > a->n_slots) return KDA_ERR_SHAPE;
  const size_t es = esize(a->io), rk = (size_t)a->Hk * a->Dk, rv = (size_t)a->Hv * a->Dv, n = (size_t)a->N;
  if (!stride_ok(a->q_stride, rk, es) || !stride_ok(a->k_stride, rk, es) || !stride_ok(a->v_stride, rv, es))
    return KDA_ERR_SHAPE;
  size_t qb, kb, vb, ob, gb, sb, wgs;
  if (!rows_bytes(qb, n, rk, a->q_stride, es) || !rows_bytes(kb, n, rk, a->k_stride, es) ||
      !rows_bytes(vb, n, rv, a->v_stride, es) || !mul_ok(ob, {n, rv, es}) || !mul_ok(gb, {n, (size_t)a->Hv, es}) ||
      !mul_ok(sb, {(size_t)a->n_slots, (size_t)a->Hv, (size_t)a->Dk, (size_t)a->Dv, 4}) ||
      !mul_ok(wgs, {n, (size_t)a->Hv}) || wgs > kGdrMaxGroups)
    return KDA_ERR_SHAPE;
  if ((a->A_log == nullptr) != (a->dt_bias == nullptr)) return KDA_ERR_NULL;
  if (!a->S || (a->N > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->o))) return KDA_ERR_NULL;
  for (const void* p : std::initializer_list<const void*>{a->q, a->k, a->v, a->g, a->beta, a->A_log, a->dt_bias,
                                                          a->S, a->slots, a->o})
    if (p && !aligned16(p)) return KDA_ERR_ALIGN;
  return disjoint({span(a->o, ob), span(a->S, sb)},
                  {span(a->q, qb), span(a->k, kb), span(a->v, vb), span(a->g, gb), span(a->beta, gb),
                   span(a->A_log, (size_t)a->Hv * 4), span(a->dt_bias, (size_t)a->Hv * 4),
                   span(a->slots, n * 4)});
}

kda_status kda_gdr_decode(const kda_gdr_decode_args* a, void* stream) {
  if (kda_status e = kda_validate_gdr_decode(a); e != KDA_OK) return e;
  GdrDecodeParams p{};
  p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta;
  p.A_log = a->A_log; p.dt_bias = a->dt_bias;
  p.beta_logits = (a->flags & KDA_FLAG_BETA_LOGITS) != 0;
  p.l2 = (a->flags & KDA_FLAG_L2NORM_QK) != 0;
  p.eps = a->l2_eps; p.scale = a->scale;
  p.S = a->S; p.slots = a->slots; p.o = a->o;
  p.N = a->N; p.n_slots = a->n_slots; p.Hk = a->Hk; p.Hv = a->Hv;
  p.qs = a->q_stride > 0 ? a->q_stride : (long)a->Hk * a->Dk;
  p.ks = a->k_stride > 0 ? a->k_stride : (long)a->Hk * a->Dk;
  p.vs = a->v_stride > 0 ? a->v_stride : (long)a->Hv * a->Dv;
  return hip_status(launch_gdr_decode(p, a->Dk, a->Dv, a->io == KDA_FP32, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ------------------------------------------------------------------ pages
namespace {

kda_status pool_ok(const kda_pages_pool* p, size_t& layer, size_t& bytes) {
  if (p == nullptr || p->data == nullptr) return KDA_ERR_NULL;
  if (p->n_layers < 1 || p->n_pages < 1 || p->page_bytes < 1 || p->layer_stride < 0) return KDA_ERR_SHAPE;
  if (p->page_bytes % 16 != 0 || p->layer_stride % 16 != 0) return KDA_ERR_ALIGN;
  size_t body;
  if (!mul_ok(body, {(size_t)p->n_pages, (size_t)p->page_bytes})) return KDA_ERR_SHAPE;
  layer = p->layer_stride > 0 ? (size_t)p->layer_stride : body;
  if (layer < body) return KDA_ERR_SHAPE;
  size_t rest;
  if (!mul_ok(rest, {(size_t)p->n_layers - 1, layer})) return KDA_ERR_SHAPE;
  bytes = rest + body;
  return aligned16(p->data) ? KDA_OK : KDA_ERR_ALIGN;
}

// workspace: 256 bytes with the count, the pairs, and one number per page
struct PagesWork {
  size_t moves, marks, bytes;
};
PagesWork pages_work(int n_pages, int n) {
  const size_t cap = n > 0 ? (size_t)n : (size_t)n_pages;  // a compaction moves less than n_pages
  PagesWork w{};
  w.moves = 256;
  w.marks = round_up(w.moves + 8 * cap, 256);
  // a copy marks destinations by page, a fork lists at most n free pages
  w.bytes = round_up(w.marks + 4 * (size_t)n_pages, 256);
  return w;
}

PagesMoveParams moves_of(const kda_pages_pool* src, size_t src_layer, const kda_pages_pool* dst, size_t dst_layer,
                         char* ws, const PagesWork& w, int cap) {
  PagesMoveParams m{};
  m.src = static_cast<const char*>(src->data);
  m.dst = static_cast<char*>(dst->data);
  m.src_layer = src_layer;
  m.dst_layer = dst_layer;
  m.page_bytes = (size_t)dst->page_bytes;
  m.layers = dst->n_layers;
  m.moves = reinterpret_cast<const int*>(ws + w.moves);
  m.count = reinterpret_cast<const int*>(ws);
  m.cap = cap;
  return m;
}

bool all16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p && !aligned16(p)) return false;
  return true;
}

}  // namespace

extern "C" {

size_t kda_pages_workspace_bytes(const kda_pages_pool* pool, int32_t n) {
  size_t layer, bytes;
  if (pool_ok(pool, layer, bytes) != KDA_OK || n < 0) return 0;
  return pages_work(pool->n_pages, n).bytes;
}

kda_status kda_pages_fork(const kda_pages_pool* pool, const int32_t* refs, int32_t* refs_out,
                          const int32_t* src, int32_t* dst, int32_t n, void* ws, size_t ws_bytes,
                          void* stream) {
  size_t layer, bytes;
  if (kda_status e = pool_ok(pool, layer, bytes); e != KDA_OK) return e;
  if (n < 0) return KDA_ERR_SHAPE;
  if (!refs || !refs_out || (n > 0 && (!src || !dst))) return KDA_ERR_NULL;
  if (!all16({refs, refs_out, src, dst})) return KDA_ERR_ALIGN;
  const size_t rb = (size_t)pool->n_pages * 4, nb = (size_t)n * 4;
  const Span po = span(pool->data, bytes), rf = span(refs, rb), ro = span(refs_out, rb), sr = span(src, nb),
             ds = span(dst, nb);
  if (!same_or_disjoint(rf, ro)) return KDA_ERR_ALIAS;
  if (kda_status e = disjoint({po, ro, ds}, {sr}); e != KDA_OK) return e;
  if (overlaps(rf, po) || overlaps(rf, ds)) return KDA_ERR_ALIAS;
  const PagesWork w = pages_work(pool->n_pages, n);
  if (kda_status e = gdr_check_ws(ws, ws_bytes, w.bytes, {po, rf, ro, sr, ds}); e != KDA_OK) return e;
  char* base = static_cast<char*>(ws);
  return hip_status(launch_pages_fork(refs, refs_out, pool->n_pages, src, dst, n,
                                      reinterpret_cast<int*>(base + w.marks),
                                      moves_of(pool, layer, pool, layer, base, w, n < pool->n_pages ? n : pool->n_pages),
                                      static_cast<hipStream_t>(stream)));
}

kda_status kda_pages_free(const int32_t* refs, int32_t* refs_out, int32_t n_pages, const int32_t* pages, int32_t n,
                          void* stream) {
  if (n_pages < 1 || n < 0) return KDA_ERR_SHAPE;
  if (!refs || !refs_out || (n > 0 && !pages)) return KDA_ERR_NULL;
  if (!all16({refs, refs_out, pages})) return KDA_ERR_ALIGN;
  const size_t rb = (size_t)n_pages * 4;
  if (!same_or_disjoint(span(refs, rb), span(refs_out, rb))) return KDA_ERR_ALIAS;
  if (overlaps(span(refs_out, rb), span(pages, (size_t)n * 4))) return KDA_ERR_ALIAS;
  return hip_status(launch_pages_free(refs, refs_out, n_pages, pages, n, static_cast<hipStream_t>(stream)));
}

kda_status kda_pages_compact(const kda_pages_pool* pool, const int32_t* refs, int32_t* refs_out, int32_t* new_id,
                             int32_t* n_used, const int32_t* table, int32_t* table_out, int64_t n_table, void* ws,
                             size_t ws_bytes, void* stream) {
  size_t layer, bytes;
  if (kda_status e = pool_ok(pool, layer, bytes); e != KDA_OK) return e;
  if (n_table < 0 || n_table > (int64_t(1) << 40)) return KDA_ERR_SHAPE;
  if (!refs || !refs_out || !new_id || !n_used || (n_table > 0 && (!table || !table_out))) return KDA_ERR_NULL;
  if (!all16({refs, refs_out, new_id, n_used, table, table_out})) return KDA_ERR_ALIGN;
  const size_t rb = (size_t)pool->n_pages * 4, tb = (size_t)n_table * 4;
  const Span po = span(pool->data, bytes), rf = span(refs, rb), ro = span(refs_out, rb), ni = span(new_id, rb),
             nu = span(n_used, 4), ti = span(table, tb), to = span(table_out, tb);
  if (!same_or_disjoint(rf, ro) || !same_or_disjoint(ti, to)) return KDA_ERR_ALIAS;
  if (kda_status e = disjoint({po, ro, ni, nu, to}, {}); e != KDA_OK) return e;
  for (const Span& x : {po, ni, nu, to})
    if (overlaps(rf, x)) return KDA_ERR_ALIAS;
  for (const Span& x : {po, ro, ni, nu})
    if (overlaps(ti, x)) return KDA_ERR_ALIAS;
  const PagesWork w = pages_work(pool->n_pages, 0);
  if (kda_status e = gdr_check_ws(ws, ws_bytes, w.bytes, {po, rf, ro, ni, nu, ti, to}); e != KDA_OK) return e;
  PagesMoveParams m = moves_of(pool, layer, pool, layer, static_cast<char*>(ws), w, pool->n_pages / 2);
  m.table = table;
  m.table_out = table_out;
  m.new_id = new_id;
  m.n_table = n_table;
  m.n_pages = pool->n_pages;
  return hip_status(launch_pages_compact(refs, refs_out, pool->n_pages, new_id, n_used, m,
                                         static_cast<hipStream_t>(stream)));
}

kda_status kda_pages_copy(const kda_pages_pool* src_pool, const kda_pages_pool* dst_pool, const int32_t* src,
                          const int32_t* dst, int32_t* done, int32_t n, void* ws, size_t ws_bytes, void* stream) {
  size_t sl, sb, dl, db;
  if (kda_status e = pool_ok(src_pool, sl, sb); e != KDA_OK) return e;
  if (kda_status e = pool_ok(dst_pool, dl, db); e != KDA_OK) return e;
  if (n < 0 || src_pool->n_layers != dst_pool->n_layers || src_pool->page_bytes != dst_pool->page_bytes)
    return KDA_ERR_SHAPE;
  if (n > 0 && (!src || !dst)) return KDA_ERR_NULL;
  if (!all16({src, dst, done})) return KDA_ERR_ALIGN;
  const Span ps = span(src_pool->data, sb), pd = span(dst_pool->data, db), sr = span(src, (size_t)n * 4),
             ds = span(dst, (size_t)n * 4), dn = span(done, (size_t)n * 4);
  const bool same = src_pool->data == dst_pool->data;
  if (same ? (src_pool->n_pages != dst_pool->n_pages || sl != dl) : overlaps(ps, pd)) return KDA_ERR_ALIAS;
  if (kda_status e = disjoint({pd, dn}, {sr, ds}); e != KDA_OK) return e;
  if (overlaps(dn, ps)) return KDA_ERR_ALIAS;
  const PagesWork w = pages_work(dst_pool->n_pages, n);
  if (kda_status e = gdr_check_ws(ws, ws_bytes, w.bytes, {ps, pd, sr, ds, dn}); e != KDA_OK) return e;
  if (n == 0) return KDA_OK;
  char* base = static_cast<char*>(ws);
  return hip_status(launch_pages_copy(src, dst, n, src_pool->n_pages, dst_pool->n_pages, same ? 1 : 0,
                                      reinterpret_cast<int*>(base + w.marks), done,
                                      moves_of(src_pool, sl, dst_pool, dl, base, w, n),
                                      static_cast<hipStream_t>(stream)));
}

}  // extern "C"
