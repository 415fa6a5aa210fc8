// decay_abi.cu -- C entry points of the linear attention with a decay per head and of layer norm:
// validation of every argument, then the passes.
#include <math.h>
#include <stdint.h>

#include "abi_rows.h"
#include "lizard_internal.h"

namespace {

using namespace lz::abi;

// (The last chunk's end, past L, is an int32 in the kernels.)
bool decay_dims_ok(const lizard_decay_dims* d) {
  return d && d->B >= 1 && d->B <= 65535 && d->H >= 1 && d->Hk >= 1 && d->H % d->Hk == 0 && d->L >= 0 &&
         dtype_ok(d->dtype) && isfinite(d->scale) && (__int128)d->B * d->H < (1 << 28) &&
         (__int128)d->B * d->H * d->L < (1ll << 31) && d->L < INT32_MAX - lz::kDecayTile;
}
bool width_ok(int d) { return d == 64 || d == 128; }

float scale_of(const lizard_decay_dims& d) { return d.scale > 0.f ? d.scale : 1.0f / sqrtf((float)d.dk); }

// Decays are read one by one: any fp32 address will do (a slice of a longer row).
bool decay_ptr_ok(const float* p, bool optional) {
  return p ? (reinterpret_cast<uintptr_t>(p) & 3u) == 0 : optional;
}

// The decays' strides and the bytes they span.
struct Decays {
  lz::Strides s{};
  size_t bytes = 0;
  bool ok = false;
};
Decays decays_of(const lizard_strides* s, int64_t B, int64_t H, int64_t L) {
  Decays r;
  r.s = s ? lz::Strides{s->n, s->h, s->t} : lz::Strides{H * L, L, 1};
  const int64_t dim[3] = {B, H, L}, st[3] = {r.s.n, r.s.h, r.s.t};
  __int128 span = 1;
  for (int i = 0; i < 3; ++i) {
    if (dim[i] <= 1) continue;
    if (st[i] < 0 || st[i] > kMaxExtent) return r;
    span += (dim[i] - 1) * (__int128)st[i];
  }
  if (span > kMaxExtent) return r;
  r.bytes = L ? (size_t)span * sizeof(float) : 0;
  r.ok = true;
  return r;
}

// Scratch of a backward call after the header.
struct BwdScratch {
  size_t dots, parts, edge, through, segs, bytes;  // offsets, then the size
};
size_t seg_bytes(const lizard_decay_dims& d, int da, int dc) {
  const size_t n = lz::decay_f32_workspace(d.B, d.H, d.L, da, dc);
  return lz::align_up(d.dtype == LIZARD_BF16 ? std::max(n, lz::decay_tc_workspace(d.B, d.H, d.L, da, dc)) : n, 256);
}
// Planes of [B,H,L] sums for d log_decay: within chunks, and with the states (the tensor-core pass
// leaves two for each 64 channels), of the rows and of the columns.  States that enter chunks: of 64 tokens,
// as the pass takes them that any strides can go to.
size_t in_planes(const lizard_decay_dims& d) { return d.dk / lz::kDecaySlice; }
size_t out_planes(const lizard_decay_dims& d) { return 2 * in_planes(d); }
size_t edge_parts(const lizard_decay_dims& d) { return lz::kDecayEdgeWarps * in_planes(d); }
BwdScratch bwd_scratch(const lizard_decay_dims& d) {
  BwdScratch w;
  const size_t rows = (size_t)d.B * d.H * d.L;
  const size_t chunks = (size_t)d.B * d.H * ((d.L + lz::kDecayChunk - 1) / lz::kDecayChunk);
  size_t at = 0;
  w.dots = at, at += lz::align_up((in_planes(d) + 2 * out_planes(d)) * rows * sizeof(float), 256);
  w.parts = at, at += d.H > d.Hk ? lz::align_up(rows * (d.dk > d.dv ? d.dk : d.dv) * sizeof(float), 256) : 0;
  w.edge = at, at += chunks * d.dk * d.dv * sizeof(float);  // a multiple of 16 KB
  w.through = at, at += lz::align_up(chunks * edge_parts(d) * sizeof(float), 256);
  w.segs = at, at += std::max(seg_bytes(d, d.dk, d.dv), seg_bytes(d, d.dv, d.dk));
  w.bytes = at;
  return w;
}

// Whether the tensor cores take rows of these strides (all of a call's, or none).
bool tc_rows(const lizard_decay_dims& d, const Tensor* t, int n) {
  if (d.dtype != LIZARD_BF16 || d.L == 0 || !lz::tma_encode_available()) return false;
  for (int i = 0; i < n; ++i)
    if (!lz::decay_tc_rows_ok((int)t[i].N, (int)t[i].H, (int)t[i].T, (int)t[i].d, t[i].r->s)) return false;
  return true;
}

bool norm_dims_ok(const lizard_norm_dims* d) {
  return d && d->N >= 1 && d->H >= 1 && d->T >= 0 && (d->per_head == 0 || d->per_head == 1) && dtype_ok(d->dtype) &&
         isfinite(d->eps) && (__int128)d->N * d->H * d->T < (1ll << 31) && (!d->per_head || d->H <= 65535);
}
bool norm_width_ok(int d) { return d >= 8 && d <= 16384 && d % 8 == 0; }

}  // namespace

extern "C" {

size_t lizard_decay_attn_workspace_bytes(const lizard_decay_dims* dims, int32_t is_bwd) {
  if (!decay_dims_ok(dims) || !width_ok(dims->dk) || !width_ok(dims->dv)) return 0;
  return lz::kWsHeader + (is_bwd ? bwd_scratch(*dims).bytes : seg_bytes(*dims, dims->dk, dims->dv));
}

lizard_status lizard_decay_attn_fwd(const lizard_decay_dims* dims, const void* q, const lizard_strides* s_q,
                                    const void* k, const lizard_strides* s_k, const void* v,
                                    const lizard_strides* s_v, const float* log_decay,
                                    const lizard_strides* s_decay, const int32_t* count, const float* h0, void* y,
                                    const lizard_strides* s_y, float* h_final, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  lz::set_last_launches(0);
  if (!decay_dims_ok(dims)) return LIZARD_ERR_INVALID_ARG;
  const lizard_decay_dims& d = *dims;
  if (!width_ok(d.dk) || !width_ok(d.dv)) return LIZARD_ERR_UNSUPPORTED;
  const bool none = d.L == 0;
  if (!ptr_ok(q, none) || !ptr_ok(k, none) || !ptr_ok(v, none) || !decay_ptr_ok(log_decay, none) || !ptr_ok(y, none) ||
      !ptr_ok(count, true) || !ptr_ok(h0, true) || !ptr_ok(h_final, true))
    return LIZARD_ERR_INVALID_ARG;
  const Rows rq = rows_of(s_q, d.B, d.H, d.L, d.dk, d.dtype, false);
  const Rows rk = rows_of(s_k, d.B, d.Hk, d.L, d.dk, d.dtype, false);
  const Rows rv = rows_of(s_v, d.B, d.Hk, d.L, d.dv, d.dtype, false);
  const Rows ry = rows_of(s_y, d.B, d.H, d.L, d.dv, d.dtype, true);
  const Decays rg = decays_of(s_decay, d.B, d.H, d.L);
  if (!rq.ok || !rk.ok || !rv.ok || !ry.ok || !rg.ok) return LIZARD_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < lizard_decay_attn_workspace_bytes(dims, 0))
    return LIZARD_ERR_WORKSPACE;
  const int64_t es = (int64_t)elem_size(d.dtype);
  const size_t states = (size_t)d.B * d.H * d.dk * d.dv * sizeof(float);
  const Span outs[] = {{h_final, states}, {workspace, workspace_bytes}};
  const Span rows[] = {{q, rq.bytes}, {k, rk.bytes}, {v, rv.bytes}, {y, ry.bytes}};
  const Span ins[] = {{log_decay, rg.bytes}, {count, (size_t)d.B * 4}, {h0, states}};
  const Tensor ty{y, &ry, d.B, d.H, d.L, d.dv, es}, tq{q, &rq, d.B, d.H, d.L, d.dk, es};
  const Tensor tk{k, &rk, d.B, d.Hk, d.L, d.dk, es}, tv{v, &rv, d.B, d.Hk, d.L, d.dv, es};
  if (any_overlap(outs, 2, rows, 4) || any_overlap(outs, 2, ins, 3) || any_overlap(rows + 3, 1, ins, 3) ||
      !apart(ty, tq) || !apart(ty, tk) || !apart(ty, tv))
    return LIZARD_ERR_INVALID_ARG;
  if (none && !h_final) return LIZARD_OK;
  const int G = d.H / d.Hk;
  lz::DecayPass a{};
  a.B = d.B, a.H = d.H, a.L = d.L, a.da = d.dk, a.dc = d.dv;
  a.a = q, a.b = k, a.c = v, a.sa = rq.s, a.sb = rk.s, a.sc = rv.s, a.ga = 1, a.gb = G, a.gc = G;
  a.lg = log_decay, a.sg = rg.s, a.count = count;
  a.init = h0, a.fin = h_final;
  a.out = y, a.so = ry.s;
  a.scale_out = scale_of(d), a.scale_in = 1.f;
  a.status = static_cast<unsigned*>(workspace);
  int launches = 0;
  const cudaStream_t s = (cudaStream_t)stream;
  const Tensor in[] = {tq, tk, tv};
  float* segs = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + lz::kWsHeader);
  if (!none && d.L <= (d.dtype == LIZARD_F32 ? lz::kDecayFewF32 : lz::kDecayFew)) {
    lz::DecayStep t{};
    t.B = d.B, t.H = d.H, t.G = G, t.L = d.L, t.dk = d.dk, t.dv = d.dv;
    t.q = q, t.k = k, t.v = v, t.sq = rq.s, t.sk = rk.s, t.sv = rv.s;
    t.lg = log_decay, t.sg = rg.s, t.count = count, t.h_in = h0, t.h_out = h_final;
    t.y = y, t.sy = ry.s, t.scale = a.scale_out, t.status = a.status;
    return finish(lz::launch_decay_step(t, d.dtype, s, &launches), launches);
  }
  const cudaError_t e = tc_rows(d, in, 3) ? lz::launch_decay_tc(a, false, segs, s, &launches)
                                          : lz::launch_decay_f32(a, d.dtype, segs, s, &launches);
  return finish(e, launches);
}

lizard_status lizard_decay_attn_bwd(const lizard_decay_dims* dims, const void* q, const lizard_strides* s_q,
                                    const void* k, const lizard_strides* s_k, const void* v,
                                    const lizard_strides* s_v, const float* log_decay,
                                    const lizard_strides* s_decay, const int32_t* count, const float* h0,
                                    const void* dy, const lizard_strides* s_dy, const float* d_h_final, void* d_q,
                                    const lizard_strides* s_dq, void* d_k, const lizard_strides* s_dk, void* d_v,
                                    const lizard_strides* s_dv, float* d_log_decay, float* d_h0, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  lz::set_last_launches(0);
  if (!decay_dims_ok(dims)) return LIZARD_ERR_INVALID_ARG;
  const lizard_decay_dims& d = *dims;
  if (!width_ok(d.dk) || !width_ok(d.dv)) return LIZARD_ERR_UNSUPPORTED;
  const bool none = d.L == 0;
  if (!ptr_ok(q, none) || !ptr_ok(k, none) || !ptr_ok(v, none) || !decay_ptr_ok(log_decay, none) || !ptr_ok(dy, none) ||
      !ptr_ok(d_q, none) || !ptr_ok(d_k, none) || !ptr_ok(d_v, none) || !ptr_ok(count, true) || !ptr_ok(h0, true) ||
      !ptr_ok(d_h_final, true) || !ptr_ok(d_log_decay, true) || !ptr_ok(d_h0, true))
    return LIZARD_ERR_INVALID_ARG;
  const Rows rq = rows_of(s_q, d.B, d.H, d.L, d.dk, d.dtype, false);
  const Rows rk = rows_of(s_k, d.B, d.Hk, d.L, d.dk, d.dtype, false);
  const Rows rv = rows_of(s_v, d.B, d.Hk, d.L, d.dv, d.dtype, false);
  const Rows ry = rows_of(s_dy, d.B, d.H, d.L, d.dv, d.dtype, false);
  const Rows oq = rows_of(s_dq, d.B, d.H, d.L, d.dk, d.dtype, true);
  const Rows ok = rows_of(s_dk, d.B, d.Hk, d.L, d.dk, d.dtype, true);
  const Rows ov = rows_of(s_dv, d.B, d.Hk, d.L, d.dv, d.dtype, true);
  const Decays rg = decays_of(s_decay, d.B, d.H, d.L);
  if (!rq.ok || !rk.ok || !rv.ok || !ry.ok || !oq.ok || !ok.ok || !ov.ok || !rg.ok) return LIZARD_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < lizard_decay_attn_workspace_bytes(dims, 1))
    return LIZARD_ERR_WORKSPACE;
  const int64_t es = (int64_t)elem_size(d.dtype);
  const size_t states = (size_t)d.B * d.H * d.dk * d.dv * sizeof(float);
  const Span flat[] = {{d_log_decay, (size_t)d.B * d.H * d.L * 4}, {d_h0, states}, {workspace, workspace_bytes}};
  const Span rows[] = {{q, rq.bytes},   {k, rk.bytes},   {v, rv.bytes},  {dy, ry.bytes},
                       {d_q, oq.bytes}, {d_k, ok.bytes}, {d_v, ov.bytes}};
  const Span ins[] = {{log_decay, rg.bytes}, {count, (size_t)d.B * 4}, {h0, states}, {d_h_final, states}};
  const Tensor in[] = {{q, &rq, d.B, d.H, d.L, d.dk, es},
                       {k, &rk, d.B, d.Hk, d.L, d.dk, es},
                       {v, &rv, d.B, d.Hk, d.L, d.dv, es},
                       {dy, &ry, d.B, d.H, d.L, d.dv, es}};
  const Tensor out[] = {{d_q, &oq, d.B, d.H, d.L, d.dk, es},
                        {d_k, &ok, d.B, d.Hk, d.L, d.dk, es},
                        {d_v, &ov, d.B, d.Hk, d.L, d.dv, es}};
  if (any_overlap(flat, 3, rows, 7) || any_overlap(flat, 3, ins, 4)) return LIZARD_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    const Span s{out[i].p, out[i].r->bytes};
    for (const Span& x : ins)
      if (overlap(s, x)) return LIZARD_ERR_INVALID_ARG;
    for (const Tensor& x : in)
      if (!apart(out[i], x)) return LIZARD_ERR_INVALID_ARG;
    for (int j = i + 1; j < 3; ++j)
      if (!apart(out[i], out[j])) return LIZARD_ERR_INVALID_ARG;
  }
  if (none && !d_h0) return LIZARD_OK;
  const int G = d.H / d.Hk;
  const float scale = scale_of(d);
  const BwdScratch w = bwd_scratch(d);
  unsigned char* ws = static_cast<unsigned char*>(workspace) + lz::kWsHeader;
  const size_t plane = (size_t)d.B * d.H * d.L;
  float* dots = reinterpret_cast<float*>(ws + w.dots);
  float *inside = dots, *row_out = inside + in_planes(d) * plane, *col_out = row_out + out_planes(d) * plane;
  float *edge = reinterpret_cast<float*>(ws + w.edge), *through = reinterpret_cast<float*>(ws + w.through);
  float* segs = reinterpret_cast<float*>(ws + w.segs);
  float* part = reinterpret_cast<float*>(ws + w.parts);
  const cudaStream_t s = (cudaStream_t)stream;
  const bool gate = d_log_decay && !none;
  const bool tc = tc_rows(d, in, 4);
  int launches = 0;
  // the gradient of log_decay takes the products with the states as results: from exact states
  auto pass = [&](const lz::DecayPass& p) {
    return tc ? lz::launch_decay_tc(p, p.x != nullptr, segs, s, &launches)
              : lz::launch_decay_f32(p, d.dtype, segs, s, &launches);
  };
  lz::DecayPass a{};
  a.B = d.B, a.H = d.H, a.L = d.L, a.lg = log_decay, a.sg = rg.s, a.count = count;
  a.status = static_cast<unsigned*>(workspace);
  // d_v: (k, q, dy) reversed; its state is dh, and leaves as d_h0
  lz::DecayPass b = a;
  b.da = d.dk, b.dc = d.dv, b.rev = true;
  b.a = k, b.b = q, b.c = dy, b.sa = rk.s, b.sb = rq.s, b.sc = ry.s, b.ga = G, b.gb = b.gc = 1;
  b.init = d_h_final, b.fin = d_h0;
  b.scale_out = 1.f, b.scale_in = scale;
  const lz::Strides heads_v{(int64_t)d.H * d.L * d.dv, (int64_t)d.L * d.dv, d.dv};
  b.out = G > 1 ? static_cast<void*>(part) : d_v, b.so = G > 1 ? heads_v : ov.s, b.out_f32 = G > 1;
  cudaError_t e = pass(b);
  if (e != cudaSuccess || none) return finish(e, launches);
  if (G > 1) e = lz::launch_decay_heads(d.B, d.Hk, G, d.L, d.dv, part, d_v, ov.s, d.dtype, s, &launches);
  if (e != cudaSuccess) return finish(e, launches);
  // d_k: (v, dy, q) reversed; its state is dh transposed
  b = a;
  b.da = d.dv, b.dc = d.dk, b.rev = true;
  b.a = v, b.b = dy, b.c = q, b.sa = rv.s, b.sb = ry.s, b.sc = rq.s, b.ga = G, b.gb = b.gc = 1;
  b.init = d_h_final, b.state_t = true;
  b.scale_out = 1.f, b.scale_in = scale;
  const lz::Strides heads_k{(int64_t)d.H * d.L * d.dk, (int64_t)d.L * d.dk, d.dk};
  b.out = G > 1 ? static_cast<void*>(part) : d_k, b.so = G > 1 ? heads_k : ok.s, b.out_f32 = G > 1;
  if (gate) b.x = k, b.sx = rk.s, b.gx = G, b.dot_out = col_out, b.edge = edge;
  e = pass(b);
  if (e == cudaSuccess && G > 1)
    e = lz::launch_decay_heads(d.B, d.Hk, G, d.L, d.dk, part, d_k, ok.s, d.dtype, s, &launches);
  if (e != cudaSuccess) return finish(e, launches);
  // d_q: (dy, v, k) forward; its state is h transposed
  b = a;
  b.da = d.dv, b.dc = d.dk;
  b.a = dy, b.b = v, b.c = k, b.sa = ry.s, b.sb = rv.s, b.sc = rk.s, b.ga = 1, b.gb = b.gc = G;
  b.init = h0, b.state_t = true;
  b.scale_out = scale, b.scale_in = 1.f;
  b.out = d_q, b.so = oq.s;
  if (gate) b.x = q, b.sx = rq.s, b.gx = 1, b.dot_in = inside, b.dot_out = row_out, b.edge = edge, b.through = through;
  e = pass(b);
  if (e != cudaSuccess || !gate) return finish(e, launches);
  if (tc) {
    lz::DecayPairs pr{};
    pr.B = d.B, pr.H = d.H, pr.G = G, pr.L = d.L, pr.dk = d.dk, pr.dv = d.dv;
    pr.q = q, pr.k = k, pr.v = v, pr.dy = dy, pr.sq = rq.s, pr.sk = rk.s, pr.sv = rv.s, pr.sy = ry.s;
    pr.lg = log_decay, pr.sg = rg.s, pr.count = count, pr.scale = scale;
    pr.inside = inside, pr.status = a.status;
    e = lz::launch_decay_pairs(pr, s, &launches);
    if (e != cudaSuccess) return finish(e, launches);
  }
  lz::DecayGate g{};
  g.B = d.B, g.H = d.H, g.L = d.L, g.chunk = tc ? lz::kDecayTile : lz::kDecayChunk;
  g.in_slices = tc ? 1 : (int)in_planes(d), g.out_slices = (int)(tc ? out_planes(d) : in_planes(d));
  g.parts = (int)edge_parts(d);
  g.inside = inside, g.row_out = row_out, g.col_out = col_out, g.through = through;
  g.count = count, g.d_lg = d_log_decay;
  e = lz::launch_decay_gate(g, s, &launches);
  return finish(e, launches);
}

lizard_status lizard_decay_attn_step(const lizard_decay_dims* dims, const void* q, const lizard_strides* s_q,
                                     const void* k, const lizard_strides* s_k, const void* v,
                                     const lizard_strides* s_v, const float* log_decay,
                                     const lizard_strides* s_decay, float* h, void* y, const lizard_strides* s_y,
                                     void* stream) {
  lz::set_last_launches(0);
  if (!decay_dims_ok(dims)) return LIZARD_ERR_INVALID_ARG;
  const lizard_decay_dims& d = *dims;
  if (!width_ok(d.dk) || !width_ok(d.dv)) return LIZARD_ERR_UNSUPPORTED;
  const bool none = d.L == 0;
  if (!ptr_ok(q, none) || !ptr_ok(k, none) || !ptr_ok(v, none) || !decay_ptr_ok(log_decay, none) || !ptr_ok(y, none) ||
      !ptr_ok(h, none))
    return LIZARD_ERR_INVALID_ARG;
  const Rows rq = rows_of(s_q, d.B, d.H, d.L, d.dk, d.dtype, false);
  const Rows rk = rows_of(s_k, d.B, d.Hk, d.L, d.dk, d.dtype, false);
  const Rows rv = rows_of(s_v, d.B, d.Hk, d.L, d.dv, d.dtype, false);
  const Rows ry = rows_of(s_y, d.B, d.H, d.L, d.dv, d.dtype, true);
  const Decays rg = decays_of(s_decay, d.B, d.H, d.L);
  if (!rq.ok || !rk.ok || !rv.ok || !ry.ok || !rg.ok) return LIZARD_ERR_INVALID_ARG;
  const int64_t es = (int64_t)elem_size(d.dtype);
  const Span outs[] = {{h, (size_t)d.B * d.H * d.dk * d.dv * sizeof(float)}};
  const Span rows[] = {{q, rq.bytes}, {k, rk.bytes}, {v, rv.bytes}, {y, ry.bytes}, {log_decay, rg.bytes}};
  const Tensor ty{y, &ry, d.B, d.H, d.L, d.dv, es}, tq{q, &rq, d.B, d.H, d.L, d.dk, es};
  const Tensor tk{k, &rk, d.B, d.Hk, d.L, d.dk, es}, tv{v, &rv, d.B, d.Hk, d.L, d.dv, es};
  if (any_overlap(outs, 1, rows, 5) || overlap(rows[3], rows[4]) || !apart(ty, tq) || !apart(ty, tk) ||
      !apart(ty, tv))
    return LIZARD_ERR_INVALID_ARG;
  if (none) return LIZARD_OK;
  lz::DecayStep a{};
  a.B = d.B, a.H = d.H, a.G = d.H / d.Hk, a.L = d.L, a.dk = d.dk, a.dv = d.dv;
  a.q = q, a.k = k, a.v = v, a.sq = rq.s, a.sk = rk.s, a.sv = rv.s;
  a.lg = log_decay, a.sg = rg.s, a.h_in = a.h_out = h, a.y = y, a.sy = ry.s, a.scale = scale_of(d);
  int launches = 0;
  const cudaError_t e = lz::launch_decay_step(a, d.dtype, (cudaStream_t)stream, &launches);
  return finish(e, launches);
}

size_t lizard_layer_norm_workspace_bytes(const lizard_norm_dims* dims) {
  if (!norm_dims_ok(dims) || !norm_width_ok(dims->d)) return 0;
  return lz::kWsHeader +
         lz::norm_part_floats(dims->N, dims->H, dims->T, dims->d, dims->per_head != 0, dims->dtype) * sizeof(float);
}

lizard_status lizard_layer_norm_fwd(const lizard_norm_dims* dims, const void* x, const lizard_strides* s_x,
                                    const void* weight, const void* bias, void* y, const lizard_strides* s_y,
                                    void* stream) {
  lz::set_last_launches(0);
  if (!norm_dims_ok(dims)) return LIZARD_ERR_INVALID_ARG;
  const lizard_norm_dims& d = *dims;
  if (!norm_width_ok(d.d)) return LIZARD_ERR_UNSUPPORTED;
  const bool none = d.T == 0;
  if (!ptr_ok(x, none) || !ptr_ok(y, none) || !ptr_ok(weight, true) || !ptr_ok(bias, true))
    return LIZARD_ERR_INVALID_ARG;
  const Rows rx = rows_of(s_x, d.N, d.H, d.T, d.d, d.dtype, false);
  const Rows ry = rows_of(s_y, d.N, d.H, d.T, d.d, d.dtype, true);
  if (!rx.ok || !ry.ok) return LIZARD_ERR_INVALID_ARG;
  const int64_t es = (int64_t)elem_size(d.dtype);
  const size_t wb = (size_t)(d.per_head ? d.H : 1) * d.d * es;
  const Span out[] = {{y, ry.bytes}}, ins[] = {{weight, wb}, {bias, wb}};
  const Tensor tx{x, &rx, d.N, d.H, d.T, d.d, es}, ty{y, &ry, d.N, d.H, d.T, d.d, es};
  const bool place = x == y && same(rx.s, ry.s);
  if (any_overlap(out, 1, ins, 2) || (!place && !apart(ty, tx))) return LIZARD_ERR_INVALID_ARG;
  if (none) return LIZARD_OK;
  lz::NormCall a{};
  a.N = d.N, a.H = d.H, a.T = d.T, a.d = d.d, a.per_head = d.per_head != 0, a.eps = d.eps > 0.f ? d.eps : 1e-5f;
  a.x = x, a.w = weight, a.b = bias, a.y = y, a.sx = rx.s, a.sy = ry.s;
  int launches = 0;
  const cudaError_t e = lz::launch_norm_fwd(a, d.dtype, (cudaStream_t)stream, &launches);
  return finish(e, launches);
}

lizard_status lizard_layer_norm_bwd(const lizard_norm_dims* dims, const void* x, const lizard_strides* s_x,
                                    const void* weight, const void* dy, const lizard_strides* s_dy, void* d_x,
                                    const lizard_strides* s_dx, float* d_weight, float* d_bias, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  lz::set_last_launches(0);
  if (!norm_dims_ok(dims)) return LIZARD_ERR_INVALID_ARG;
  const lizard_norm_dims& d = *dims;
  if (!norm_width_ok(d.d)) return LIZARD_ERR_UNSUPPORTED;
  const bool none = d.T == 0;
  if (!ptr_ok(x, none) || !ptr_ok(dy, none) || !ptr_ok(d_x, true) || !ptr_ok(weight, true) ||
      !ptr_ok(d_weight, true) || !ptr_ok(d_bias, true))
    return LIZARD_ERR_INVALID_ARG;
  const Rows rx = rows_of(s_x, d.N, d.H, d.T, d.d, d.dtype, false);
  const Rows ry = rows_of(s_dy, d.N, d.H, d.T, d.d, d.dtype, false);
  const Rows ro = rows_of(s_dx, d.N, d.H, d.T, d.d, d.dtype, true);
  if (!rx.ok || !ry.ok || !ro.ok) return LIZARD_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < lizard_layer_norm_workspace_bytes(dims))
    return LIZARD_ERR_WORKSPACE;
  const int64_t es = (int64_t)elem_size(d.dtype);
  const size_t w = (size_t)(d.per_head ? d.H : 1) * d.d;
  const Span flat[] = {{d_weight, w * 4}, {d_bias, w * 4}, {workspace, workspace_bytes}};
  const Span rows[] = {{x, rx.bytes}, {dy, ry.bytes}, {d_x, ro.bytes}, {weight, w * es}};
  const Tensor tx{x, &rx, d.N, d.H, d.T, d.d, es}, ty{dy, &ry, d.N, d.H, d.T, d.d, es};
  const Tensor to{d_x, &ro, d.N, d.H, d.T, d.d, es};
  const bool on_x = d_x == x && same(ro.s, rx.s), on_dy = d_x == dy && same(ro.s, ry.s);
  if (any_overlap(flat, 3, rows, 4) || overlap(rows[2], rows[3]) || (d_x && !on_x && !apart(to, tx)) ||
      (d_x && !on_dy && !apart(to, ty)))
    return LIZARD_ERR_INVALID_ARG;
  if (!d_x && !d_weight && !d_bias) return LIZARD_OK;
  const cudaStream_t s = (cudaStream_t)stream;
  if (none) {
    cudaError_t e = cudaSuccess;
    for (float* p : {d_weight, d_bias})
      if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, w * sizeof(float), s);
    return finish(e, 0);
  }
  lz::NormCall a{};
  a.N = d.N, a.H = d.H, a.T = d.T, a.d = d.d, a.per_head = d.per_head != 0, a.eps = d.eps > 0.f ? d.eps : 1e-5f;
  a.x = x, a.w = weight, a.dy = dy, a.y = d_x, a.sx = rx.s, a.sdy = ry.s, a.sy = ro.s;
  a.dw = d_weight, a.db = d_bias;
  if (d_weight || d_bias) a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + lz::kWsHeader);
  int launches = 0;
  const cudaError_t e = lz::launch_norm_bwd(a, d.dtype, s, &launches);
  return finish(e, launches);
}

}  // extern "C"
