// cache_abi.cu -- C entry points of the rotary positions, the 8-bit paged cache and the
// attention over it: validation of every argument, then one launcher call.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "abi_rows.h"
#include "lizard_internal.h"

namespace {

using namespace lz::abi;

// null `rope` means no rotation.
bool rope_ok(const lizard_rope* rope, int d, lz::RopeArgs* out) {
  *out = lz::RopeArgs{nullptr, 0, 0, 1.f};
  if (!rope) return true;
  if (!ptr_ok(rope->turns, false) || rope->rot < 2 || rope->rot > d || rope->rot % 2) return false;
  if (rope->layout != LIZARD_ROPE_HALF && rope->layout != LIZARD_ROPE_INTERLEAVED) return false;
  if (!(rope->attn_factor > 0.f) || !isfinite(rope->attn_factor)) return false;
  *out = lz::RopeArgs{rope->turns, rope->rot, rope->layout, rope->attn_factor};
  return true;
}

lizard_status cache_ok(const lizard_cache* c, lz::CacheArgs* out) {
  if (!c || c->N < 1 || c->N > 65535 || c->max_pages < 1 || c->pages < 1 || c->Hk < 1 || c->Hk > 32767)
    return LIZARD_ERR_INVALID_ARG;
  if (c->format != LIZARD_KV_E4M3 && c->format != LIZARD_KV_I8) return LIZARD_ERR_INVALID_ARG;
  if (!ptr_ok(c->k_codes, false) || !ptr_ok(c->v_codes, false) || !ptr_ok(c->k_scale, false) ||
      !ptr_ok(c->v_scale, false) || !ptr_ok(c->table, false))
    return LIZARD_ERR_INVALID_ARG;
  const int P = c->page_tokens;
  if ((c->d != 64 && c->d != 128) || (P != 16 && P != 32 && P != 64 && P != 128))
    return LIZARD_ERR_UNSUPPORTED;
  if ((__int128)c->pages * c->Hk * P * c->d > kMaxExtent || 
      (__int128)c->pages * c->Hk * P >= (1ll << 35) || (int64_t)c->max_pages * P > (1ll << 30))
    return LIZARD_ERR_INVALID_ARG;
  *out = lz::CacheArgs{static_cast<unsigned char*>(c->k_codes), static_cast<unsigned char*>(c->v_codes),
                       c->k_scale, c->v_scale, c->table, c->N, c->max_pages, c->pages, c->Hk, P,
                       P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7, c->d, (int)c->format};
  return LIZARD_OK;
}

// The cache's five buffers as spans: codes and scales, then the table.
void cache_spans(const lz::CacheArgs& c, Span (&s)[5]) {
  const size_t codes = (size_t)c.pages * c.Hk * c.P * c.d, scales = (size_t)c.pages * c.Hk * sizeof(float);
  s[0] = {c.k, codes}, s[1] = {c.v, codes}, s[2] = {c.ks, scales}, s[3] = {c.vs, scales};
  s[4] = {c.table, (size_t)c.N * c.max_pages * sizeof(int32_t)};
}

lizard_status rope_call(const lizard_rope_dims* dims, const lizard_rope* rope, float sign, const void* x_q,
                        const lizard_strides* s_xq, const void* x_k, const lizard_strides* s_xk,
                        const int64_t* positions, void* y_q, const lizard_strides* s_yq, void* y_k,
                        const lizard_strides* s_yk, void* stream) {
  lz::set_last_launches(0);
  if (!dims || !rope) return LIZARD_ERR_INVALID_ARG;
  const lizard_rope_dims& d = *dims;
  if (d.N < 1 || d.H < 1 || d.Hk < 0 || d.T < 0 || !dtype_ok(d.dtype)) return LIZARD_ERR_INVALID_ARG;
  if (d.d < 8 || d.d > 512 || d.d % 8) return LIZARD_ERR_UNSUPPORTED;
  lz::RopeCall a{};
  if (!rope_ok(rope, d.d, &a.rope)) return LIZARD_ERR_INVALID_ARG;
  const bool keys = d.Hk > 0;
  if (!ptr_ok(x_q, d.T == 0) || !ptr_ok(y_q, d.T == 0) || !ptr_ok(positions, true))
    return LIZARD_ERR_INVALID_ARG;
  if (!ptr_ok(x_k, !keys || d.T == 0) || !ptr_ok(y_k, !keys || d.T == 0)) return LIZARD_ERR_INVALID_ARG;
  const Rows xq = rows_of(s_xq, d.N, d.H, d.T, d.d, d.dtype, false);
  const Rows yq = rows_of(s_yq, d.N, d.H, d.T, d.d, d.dtype, true);
  const Rows xk = rows_of(s_xk, d.N, d.Hk, d.T, d.d, d.dtype, false);
  const Rows yk = rows_of(s_yk, d.N, d.Hk, d.T, d.d, d.dtype, true);
  if (!xq.ok || !yq.ok || !xk.ok || !yk.ok) return LIZARD_ERR_INVALID_ARG;
  // in place means the same rows; any other overlap is refused
  const bool place_q = x_q == y_q && same(xq.s, yq.s), place_k = keys && x_k == y_k && same(xk.s, yk.s);
  const size_t npos = (size_t)d.N * d.T * sizeof(int64_t);
  const Span out_q[] = {{y_q, yq.bytes}}, out_k[] = {{keys ? y_k : nullptr, yk.bytes}};
  const Span fixed[] = {{positions, npos}, {a.rope.turns, (size_t)a.rope.rot * 4}};
  if (any_overlap(out_q, 1, fixed, 2) || any_overlap(out_k, 1, fixed, 2)) return LIZARD_ERR_INVALID_ARG;
  const int64_t es = (int64_t)elem_size(d.dtype);
  const Tensor tyq{y_q, &yq, d.N, d.H, d.T, d.d, es}, txq{x_q, &xq, d.N, d.H, d.T, d.d, es};
  const Tensor tyk{y_k, &yk, d.N, d.Hk, d.T, d.d, es}, txk{x_k, &xk, d.N, d.Hk, d.T, d.d, es};
  if (!place_q && !apart(tyq, txq)) return LIZARD_ERR_INVALID_ARG;
  if (keys && ((!place_k && !apart(tyk, txk)) || !apart(tyq, tyk) || !apart(tyq, txk) || !apart(tyk, txq)))
    return LIZARD_ERR_INVALID_ARG;
  if (d.T == 0) return LIZARD_OK;
  if ((__int128)d.N * d.T * d.d * ((int64_t)d.H + d.Hk) > kMaxExtent) return LIZARD_ERR_INVALID_ARG;
  a.N = d.N, a.H = d.H, a.Hk = d.Hk, a.T = d.T, a.d = d.d, a.sign = sign;
  a.xq = x_q, a.xk = x_k, a.yq = y_q, a.yk = y_k;
  a.sxq = xq.s, a.sxk = xk.s, a.syq = yq.s, a.syk = yk.s;
  a.positions = positions;
  int launches = 0;
  const cudaError_t e = lz::launch_rope(a, d.dtype, (cudaStream_t)stream, &launches);
  return finish(e, launches);
}

lizard_status io_call(const lizard_cache* cache, const lizard_cache_io* io, void* k,
                      const lizard_strides* s_k, void* v, const lizard_strides* s_v,
                      const lizard_rope* rope, const int64_t* pos, const int32_t* count, bool write,
                      void* workspace, size_t workspace_bytes, void* stream) {
  lz::set_last_launches(0);
  lz::CacheIo a{};
  const lizard_status st = cache_ok(cache, &a.c);
  if (st != LIZARD_OK) return st;
  if (!io || io->T < 0 || !dtype_ok(io->dtype) || !rope_ok(rope, a.c.d, &a.rope)) return LIZARD_ERR_INVALID_ARG;
  const bool none = io->T == 0;
  if (!ptr_ok(k, none) || !ptr_ok(v, none) || !ptr_ok(pos, false) || !ptr_ok(count, true))
    return LIZARD_ERR_INVALID_ARG;
  const Rows rk = rows_of(s_k, a.c.N, a.c.Hk, io->T, a.c.d, io->dtype, !write);
  const Rows rv = rows_of(s_v, a.c.N, a.c.Hk, io->T, a.c.d, io->dtype, !write);
  if (!rk.ok || !rv.ok) return LIZARD_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < lizard_cache_workspace_bytes())
    return LIZARD_ERR_WORKSPACE;
  Span c[5];
  cache_spans(a.c, c);
  const Span rows[] = {{k, rk.bytes}, {v, rv.bytes}};
  const Span small[] = {c[4], {pos, (size_t)a.c.N * 8}, {count, (size_t)a.c.N * 4},
                        {a.rope.turns, (size_t)a.rope.rot * 4}};
  const Span ws[] = {{workspace, workspace_bytes}};
  if (any_overlap(ws, 1, c, 5) || any_overlap(ws, 1, rows, 2) || any_overlap(ws, 1, small + 1, 3) ||
      any_overlap(c, 4, small, 4) || any_overlap(c, 4, rows, 2))
    return LIZARD_ERR_INVALID_ARG;
  if (!write) {  // the rows are outputs, apart from each other and from what is read
    const int64_t es = (int64_t)elem_size(io->dtype);
    const Tensor tk{k, &rk, a.c.N, a.c.Hk, io->T, a.c.d, es}, tv{v, &rv, a.c.N, a.c.Hk, io->T, a.c.d, es};
    if (any_overlap(rows, 1, small, 4) || any_overlap(rows + 1, 1, small, 4) || !apart(tk, tv))
      return LIZARD_ERR_INVALID_ARG;
  }
  if (none) return LIZARD_OK;
  a.T = io->T;
  a.k = k, a.v = v, a.sk = rk.s, a.sv = rv.s;
  a.pos = pos, a.count = count;
  a.status = static_cast<unsigned*>(workspace);
  int launches = 0;
  const cudaError_t e = write ? lz::launch_cache_write(a, io->dtype, (cudaStream_t)stream, &launches)
                              : lz::launch_cache_read(a, io->dtype, (cudaStream_t)stream, &launches);
  return finish(e, launches);
}

bool attn_dims_ok(const lz::CacheArgs& c, const lizard_cache_attn_dims* d) {
  if (!d || d->H < 1 || d->H % c.Hk || d->T < 0 || d->M < 0 || d->M > 16 || d->W < 0 || !dtype_ok(d->dtype) ||
      !isfinite(d->scale) || !isfinite(d->alpha))
    return false;
  return (__int128)c.N * d->H * d->T < (1ll << 31);
}

}  // namespace

extern "C" {

lizard_status lizard_rope_table(const lizard_rope_spec* spec, uint64_t* table) {
  if (!spec || !table) return LIZARD_ERR_INVALID_ARG;
  const lizard_rope_spec& s = *spec;
  if (s.rot < 2 || s.rot > 512 || s.rot % 2 || !(s.base > 1.0) || !isfinite(s.base)) return LIZARD_ERR_INVALID_ARG;
  if (s.scaling < LIZARD_ROPE_PLAIN || s.scaling > LIZARD_ROPE_PARTS) return LIZARD_ERR_INVALID_ARG;
  if (s.scaling != LIZARD_ROPE_PLAIN && !(s.factor >= 1.0 && isfinite(s.factor))) return LIZARD_ERR_INVALID_ARG;
  if (s.scaling == LIZARD_ROPE_PARTS &&
      !(s.low >= 0.0 && s.high > s.low && isfinite(s.high) && s.original >= 1))
    return LIZARD_ERR_INVALID_ARG;
  // extended precision: a far position multiplies the relative error of theta_i
  const long double two_pi = 6.283185307179586476925286766559L;
  for (int i = 0; i < s.rot / 2; ++i) {
    long double th = powl((long double)s.base, -2.0L * i / s.rot);
    if (s.scaling == LIZARD_ROPE_LINEAR) th /= s.factor;
    if (s.scaling == LIZARD_ROPE_PARTS) {
      const long double turns = (long double)s.original * th / two_pi;
      const long double keep = std::min(1.0L, std::max(0.0L, (turns - s.low) / ((long double)s.high - s.low)));
      th *= keep + (1.0L - keep) / s.factor;
    }
    table[i] = (uint64_t)roundl(ldexpl(th / two_pi, 64));  // below 2^64 / 6
  }
  return LIZARD_OK;
}

lizard_status lizard_rope_fwd(const lizard_rope_dims* dims, const lizard_rope* rope, const void* x_q,
                              const lizard_strides* s_xq, const void* x_k, const lizard_strides* s_xk,
                              const int64_t* positions, void* y_q, const lizard_strides* s_yq, void* y_k,
                              const lizard_strides* s_yk, void* stream) {
  return rope_call(dims, rope, 1.f, x_q, s_xq, x_k, s_xk, positions, y_q, s_yq, y_k, s_yk, stream);
}

lizard_status lizard_rope_bwd(const lizard_rope_dims* dims, const lizard_rope* rope, const void* dy_q,
                              const lizard_strides* s_dyq, const void* dy_k, const lizard_strides* s_dyk,
                              const int64_t* positions, void* dx_q, const lizard_strides* s_dxq, void* dx_k,
                              const lizard_strides* s_dxk, void* stream) {
  return rope_call(dims, rope, -1.f, dy_q, s_dyq, dy_k, s_dyk, positions, dx_q, s_dxq, dx_k, s_dxk, stream);
}

size_t lizard_cache_workspace_bytes(void) { return lz::kWsHeader; }

lizard_status lizard_cache_write(const lizard_cache* cache, const lizard_cache_io* io, const void* k,
                                 const lizard_strides* s_k, const void* v, const lizard_strides* s_v,
                                 const lizard_rope* rope, const int64_t* pos, const int32_t* count,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  return io_call(cache, io, const_cast<void*>(k), s_k, const_cast<void*>(v), s_v, rope, pos, count, true,
                 workspace, workspace_bytes, stream);
}

lizard_status lizard_cache_read(const lizard_cache* cache, const lizard_cache_io* io, const int64_t* pos,
                                const int32_t* count, void* k, const lizard_strides* s_k, void* v,
                                const lizard_strides* s_v, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return io_call(cache, io, k, s_k, v, s_v, nullptr, pos, count, false, workspace, workspace_bytes, stream);
}

size_t lizard_cache_attn_workspace_bytes(const lizard_cache* cache, const lizard_cache_attn_dims* dims) {
  lz::CacheArgs c;
  if (cache_ok(cache, &c) != LIZARD_OK || !attn_dims_ok(c, dims)) return 0;
  return lz::kWsHeader + lz::cache_attn_workspace(c.N, c.Hk, dims->H, dims->T, c.d, dims->dtype);
}

lizard_status lizard_cache_attn(const lizard_cache* cache, const lizard_cache_attn_dims* dims, const void* q,
                                const lizard_strides* s_q, const lizard_rope* rope, const int64_t* pos,
                                const int32_t* count, const int64_t* first, const void* meta_k,
                                const void* meta_v, const void* y_add, const lizard_strides* s_add, void* y,
                                const lizard_strides* s_y, void* workspace, size_t workspace_bytes,
                                void* stream) {
  lz::set_last_launches(0);
  lz::CacheAttn a{};
  const lizard_status st = cache_ok(cache, &a.c);
  if (st != LIZARD_OK) return st;
  if (!attn_dims_ok(a.c, dims) || !rope_ok(rope, a.c.d, &a.rope)) return LIZARD_ERR_INVALID_ARG;
  const lizard_cache_attn_dims& d = *dims;
  const bool none = d.T == 0;
  if (!ptr_ok(q, none) || !ptr_ok(y, none) || !ptr_ok(y_add, true) || !ptr_ok(pos, false) ||
      !ptr_ok(count, true) || !ptr_ok(first, true) || !ptr_ok(meta_k, d.M == 0) || !ptr_ok(meta_v, d.M == 0))
    return LIZARD_ERR_INVALID_ARG;
  const Rows rq = rows_of(s_q, a.c.N, d.H, d.T, a.c.d, d.dtype, false);
  const Rows ra = rows_of(s_add, a.c.N, d.H, d.T, a.c.d, d.dtype, false);
  const Rows ry = rows_of(s_y, a.c.N, d.H, d.T, a.c.d, d.dtype, true);
  if (!rq.ok || !ra.ok || !ry.ok) return LIZARD_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < lizard_cache_attn_workspace_bytes(cache, dims))
    return LIZARD_ERR_WORKSPACE;
  Span c[5];
  cache_spans(a.c, c);
  const size_t meta = (size_t)d.H * d.M * a.c.d * elem_size(d.dtype);
  const Span outs[] = {{y, ry.bytes}, {workspace, workspace_bytes}};
  const Span ins[] = {{pos, (size_t)a.c.N * 8}, {count, (size_t)a.c.N * 4}, {first, (size_t)a.c.N * 8},
                      {meta_k, meta}, {meta_v, meta}, {a.rope.turns, (size_t)a.rope.rot * 4}};
  const Span rows[] = {{q, rq.bytes}, {y_add, ra.bytes}};
  const int64_t es = (int64_t)elem_size(d.dtype);
  const Tensor tq{q, &rq, a.c.N, d.H, d.T, a.c.d, es}, ta{y_add, &ra, a.c.N, d.H, d.T, a.c.d, es};
  const Tensor ty{y, &ry, a.c.N, d.H, d.T, a.c.d, es};
  const bool place = y_add == y && same(ra.s, ry.s);
  if (any_overlap(outs, 2, ins, 6) || any_overlap(outs, 2, c, 5) || any_overlap(outs + 1, 1, rows, 2) ||
      !apart(ty, tq) || (!place && !apart(ty, ta)))
    return LIZARD_ERR_INVALID_ARG;
  if (none) return LIZARD_OK;
  a.H = d.H, a.T = d.T, a.M = d.M, a.W = d.W;
  a.scale = d.scale > 0.f ? d.scale : 1.0f / sqrtf((float)a.c.d);
  a.alpha = d.alpha;
  a.q = q, a.sq = rq.s;
  a.pos = pos, a.count = count, a.first = first;
  a.mk = meta_k, a.mv = meta_v;
  a.add = y_add, a.sadd = ra.s;
  a.y = y, a.sy = ry.s;
  a.status = static_cast<unsigned*>(workspace);
  a.ws = static_cast<unsigned char*>(workspace) + lz::kWsHeader;
  int launches = 0;
  const cudaError_t e = lz::launch_cache_attn(a, d.dtype, (cudaStream_t)stream, &launches);
  return finish(e, launches);
}

}  // extern "C"
