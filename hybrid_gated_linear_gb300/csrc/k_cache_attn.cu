// k_cache_attn.cu -- attention over the 8-bit paged cache, merged with another branch.
//
// One warp per (sequence, query head, new token): each lane holds D/32 channels of the
// query, the logits of the visible tokens come one at a time, and a running maximum m and
// sum l rescale the accumulated output (o <- o e^{m-m'} + e^{z-m'} v), so the cache is read
// once.  Meta tokens meet the query before its rotation.
#include "kv_cache.cuh"

namespace lz {
namespace {

constexpr int kWarps = 8;

template <int D, int F>
__device__ __forceinline__ void load_codes(const unsigned char* row, int r, int lane, float (&x)[D / 32]) {
  constexpr int E = D / 32;
  const int e = lane * E;
  const unsigned char* p = row + chunk_place<D>(r, e / 16) * 16 + e % 16;
  const uint32_t w = E == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
  const float4 v = codes_to_float<F>(w);
  x[0] = v.x, x[1] = v.y;
  if (E == 4) x[E - 2] = v.z, x[E - 1] = v.w;
}

template <typename T, int D, int F>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(CacheAttn a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (int64_t)a.c.N * a.H * a.T) return;
  const int t = (int)(row % a.T), h = (int)(row / a.T % a.H), n = (int)(row / a.T / a.H);
  const int hk = h / (a.H / a.c.Hk);
  T* y = static_cast<T*>(a.y) + n * a.sy.n + h * a.sy.h + t * a.sy.t;
  const int cnt = a.count ? a.count[n] : a.T;
  const int64_t p0 = a.pos[n], p = p0 + t;
  const int64_t first = a.first ? a.first[n] : 0;
  const bool known = cnt >= 0 && cnt <= a.T && p0 >= 0;
  if (!known && lane == 0) raise_status(a.status, kDevCheck);
  if (t >= cnt || cnt > a.T) {
#pragma unroll
    for (int i = 0; i < E; ++i) y[lane * E + i] = cvt_out<T>(0.f);
    return;
  }
  // the pages all of this sequence's queries see have to fit the table
  int64_t lo0 = a.W > 0 ? p0 - a.W + 1 : 0;
  lo0 = max(lo0, max(first, (int64_t)0));
  const bool seen = known && lo0 <= p0 + cnt - 1;
  const bool fits = seen && span_ok(a.c, lo0, p0 + cnt - 1);
  if (seen && !fits && lane == 0) raise_status(a.status, kDevCheck);
  const int64_t lo = max(lo0, a.W > 0 ? p - a.W + 1 : (int64_t)0);

  const T* qp = static_cast<const T*>(a.q) + n * a.sq.n + h * a.sq.h + t * a.sq.t;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) q[i] = ld_f(qp + lane * E + i), o[i] = 0.f;
  auto add = [&](float z, const float (&v)[E], float s) {
    const float mn = fmaxf(m, z);
    const float f = expf(m - mn), w = expf(z - mn);
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(w * s, v[i], o[i] * f);
    m = mn;
  };
  for (int j = 0; j < a.M; ++j) {
    const T* k = static_cast<const T*>(a.mk) + ((size_t)h * a.M + j) * D + lane * E;
    const T* v = static_cast<const T*>(a.mv) + ((size_t)h * a.M + j) * D + lane * E;
    float z = 0.f, x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) z = fmaf(q[i], ld_f(k + i), z), x[i] = ld_f(v + i);
    add(warp_sum(z) * a.scale, x, 1.f);
  }
  if (a.rope.turns) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = lane * E + i, hr = a.rope.rot / 2;
      if (e < a.rope.rot) {
        const bool half = a.rope.layout == LIZARD_ROPE_HALF;
        const bool low = half ? e < hr : e % 2 == 0;
        const int pair = half ? (low ? e : e - hr) : e / 2;
        const float other = ld_f(qp + (half ? (low ? e + hr : e - hr) : e ^ 1));
        float co, si;
        rope_angle(a.rope.turns[pair], p, a.rope.factor, co, si);
        q[i] = low ? q[i] * co - other * si : q[i] * co + other * si;
      }
    }
  }
  if (fits) {
    for (int64_t pg = lo >> a.c.log_p; pg <= p >> a.c.log_p; ++pg) {
      const int id = pool_page(a.c, n, (uint32_t)pg);
      if (id < 0) {
        if (lane == 0) raise_status(a.status, kDevCheck);
        continue;
      }
      const size_t ph = (size_t)id * a.c.Hk + hk;
      const unsigned char *kp = a.c.k + ph * a.c.P * D, *vp = a.c.v + ph * a.c.P * D;
      const float ks = a.c.ks[ph] * a.scale, vs = a.c.vs[ph];
      const int64_t t0 = pg << a.c.log_p;
      const int r0 = (int)max((int64_t)0, lo - t0), r1 = (int)min((int64_t)a.c.P - 1, p - t0);
      for (int r = r0; r <= r1; ++r) {
        float k[E], v[E], z = 0.f;
        load_codes<D, F>(kp + (size_t)r * D, r, lane, k);
        load_codes<D, F>(vp + (size_t)r * D, r, lane, v);
#pragma unroll
        for (int i = 0; i < E; ++i) z = fmaf(q[i], k[i], z);
        add(warp_sum(z) * ks, v, vs);
      }
    }
  }
  const float f = l > 0.f ? a.alpha / l : 0.f;
  const T* add_p = a.add ? static_cast<const T*>(a.add) + n * a.sadd.n + h * a.sadd.h + t * a.sadd.t : nullptr;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = lane * E + i;
    y[e] = cvt_out<T>(o[i] * f + (add_p ? ld_f(add_p + e) : 0.f));
  }
}

template <typename T, int D, int F>
cudaError_t launch(const CacheAttn& a, cudaStream_t s, int* launches) {
  const int64_t rows = (int64_t)a.c.N * a.H * a.T;
  trace_begin("cache_attn", s);
  attn_kernel<T, D, F><<<(unsigned)((rows + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a);
  trace_end(s);
  ++*launches;
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t by_format(const CacheAttn& a, cudaStream_t s, int* launches) {
  return a.c.fmt == LIZARD_KV_E4M3 ? launch<T, D, 0>(a, s, launches) : launch<T, D, 1>(a, s, launches);
}

}  // namespace

size_t cache_attn_workspace(int, int, int, int, int) { return 0; }

cudaError_t launch_cache_attn(const CacheAttn& a, lizard_dtype dt, cudaStream_t s, int* launches) {
  if (dt == LIZARD_F32)
    return a.c.d == 64 ? by_format<float, 64>(a, s, launches) : by_format<float, 128>(a, s, launches);
  return a.c.d == 64 ? by_format<bf16, 64>(a, s, launches) : by_format<bf16, 128>(a, s, launches);
}

}  // namespace lz
