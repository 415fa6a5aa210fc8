// k_cache.cu -- writing new tokens into the 8-bit paged cache and reading them back.
//
// Write.  A CTA takes a touched page of a sequence, keys or values, for one head (or kHeads, one
// after the other, where there are CTAs enough).  It holds the new rows of the page in
// registers, reduces their largest magnitude, settles the page's scale and stores the codes:
// one pass over the inputs, no second read.  The scale is a power of two, so dividing by it is
// exact, and codes of earlier tokens change only when the scale grows (they are then read,
// rescaled exactly and rounded again).
// Read.  One thread per 16 codes of a row, keys and values in one launch.
// Both are memory bound where prompts are long and bound by a chain of dependent loads
// (position, page, row) for single tokens.  Measured, 8 heads of 128, e4m3: four prompts of 4096
// tokens (100 MB each way), write 52 us with rotation and 41 without, read 18 us, back to back with
// part of the data in L2 (cold, under ncu: 56 and 22); one token of 64 sequences, write 8 us.
#include <algorithm>

#include "kv_cache.cuh"

namespace lz {
namespace {

constexpr int kThreads = 256;

// 16 consecutive elements of a row as loaded, and as floats: loads in one loop, conversions
// (the first uses, which wait) in the next.
template <typename T> struct Raw16 {
  uint4 v[sizeof(T)];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void value(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (sizeof(T) == 4) {
          x[4 * i + j] = __uint_as_float(w[j]);
        } else {
          x[(8 * i + 2 * j) & 15] = __uint_as_float(w[j] << 16);
          x[(8 * i + 2 * j + 1) & 15] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    }
  }
};

// Cosines and sines of a row's pairs in shared memory, four floats of padding every 32: lanes
// that read the pairs of different chunks with 16-byte accesses hit different banks.
__device__ __forceinline__ int pair_at(int i) { return i + 4 * (i >> 5); }
__host__ __device__ constexpr int row_floats(int pairs) { return (pairs + 4 * ((pairs - 1) >> 5) + 3) & ~3; }

// Half layout with pairs that do not come in whole chunks; kept out of line for its registers.
template <typename T>
__device__ __noinline__ void rotate_odd(int rot, const T* row, int c, const float* co, const float* si, float* x) {
  const int hr = rot / 2;
  for (int i = 0; i < 16 && c + i < rot; ++i) {
    const int e = c + i;
    const bool low = e < hr;
    const int q = pair_at(low ? e : e - hr);
    const float other = ld_f(row + (low ? e + hr : e - hr));
    x[i] = low ? x[i] * co[q] - other * si[q] : x[i] * co[q] + other * si[q];
  }
}

// Rotates channels c..c+15 (already in x, the pairs' other channels in o where they form a
// chunk too) of a row; co and si hold the row's cosines and sines.
template <typename T>
__device__ __forceinline__ void rotate16(const RopeArgs& r, const T* row, int c, const float* co, const float* si,
                                         const float (&o)[16], float (&x)[16]) {
  if (c >= r.rot) return;
  const int hr = r.rot / 2;
  if (r.layout == LIZARD_ROPE_INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 2 * i < r.rot) {
        const int q = pair_at(c / 2 + i);
        const float f = co[q], g = si[q], a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * f - b * g;
        x[2 * i + 1] = b * f + a * g;
      }
  } else if (hr % 16 == 0) {
    const float sign = c < hr ? -1.f : 1.f;
    const int q = pair_at(c < hr ? c : c - hr);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(co + q + i), g = *reinterpret_cast<const float4*>(si + q + i);
      x[i] = x[i] * f.x + sign * o[i] * g.x;
      x[i + 1] = x[i + 1] * f.y + sign * o[i + 1] * g.y;
      x[i + 2] = x[i + 2] * f.z + sign * o[i + 2] * g.z;
      x[i + 3] = x[i + 3] * f.w + sign * o[i + 3] * g.w;
    }
  } else {
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = x[i];
    rotate_odd(r.rot, row, c, co, si, y);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = y[i];
  }
}

// Heads that a CTA takes one after the other where there are CTAs enough: the next head's loads
// are in flight while this one's maximum is found and its codes are stored, and rotated keys
// share their angles.
constexpr int kHeads = 4;

// TH threads hold CH 16-channel chunks each of the new rows of a page.  One warp where they
// suffice (a decode step), so that many heads share an SM.
template <typename T, int D, int F, int CH, int TH>
__global__ void __launch_bounds__(TH, TH == 256 ? 2 : 1) write_kernel(CacheIo a, int per) {
  constexpr int C = D / 16;
  extern __shared__ __align__(16) float s_cs[];  // cosines, then sines, of every new row's pairs
  __shared__ float s_max[TH / 32];
  pdl_wait();
  const int n = blockIdx.z, tid = threadIdx.x;
  const bool values = blockIdx.y & 1;
  const int h0 = (int)(blockIdx.y >> 1) * per, h1 = min(h0 + per, a.c.Hk);
  const int64_t p0 = a.pos[n];
  const int cnt = a.count ? a.count[n] : a.T;
  if (cnt == 0) return;
  const bool bad = cnt < 0 || cnt > a.T || p0 < 0 || !span_ok(a.c, p0, last_of(p0, cnt));
  if (bad) {
    if (tid == 0) raise_status(a.status, kDevCheck);
    return;
  }
  const int64_t page = (p0 >> a.c.log_p) + blockIdx.x;
  if (page > ((p0 + cnt - 1) >> a.c.log_p)) return;
  const int id = pool_page(a.c, n, (uint32_t)page);
  if (id < 0) {
    if (tid == 0) raise_status(a.status, kDevCheck);
    return;
  }
  const int64_t t0 = page << a.c.log_p;  // position of the page's first row
  const int r0 = t0 < p0 ? (int)(p0 - t0) : 0;
  const int r1 = (int)min((int64_t)a.c.P, p0 + cnt - t0);
  const Strides st = values ? a.sv : a.sk;
  const bool turn = !values && a.rope.turns;
  const int pairs = a.rope.rot / 2, rf = row_floats(pairs);
  float* s_si = s_cs + (size_t)min(a.T, a.c.P) * rf;
  if (turn) {
    for (int e = tid; e < (r1 - r0) * pairs; e += TH) {
      const int r = e / pairs, i = e - r * pairs, q = r * rf + pair_at(i);
      rope_angle(a.rope.turns[i], t0 + r0 + r, a.rope.factor, s_cs[q], s_si[q]);
    }
    __syncthreads();
  }
  const bool chunked = turn && a.rope.layout == LIZARD_ROPE_HALF && pairs % 16 == 0;

  const T* in = static_cast<const T*>(values ? a.v : a.k) + n * st.n;
  Raw16<T> raw[CH], other[CH];
  float had = 0.f;
  auto load = [&](int hk) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int e = tid + i * TH, r = r0 + e / C, c = e % C * 16;
      if (r < r1) {
        const T* row = in + hk * st.h + (t0 + r - p0) * st.t;
        raw[i].load(row + c);
        if (chunked && c < a.rope.rot) other[i].load(row + (c < pairs ? c + pairs : c - pairs));
      }
    }
    if (r0 > 0) had = ((values ? a.c.vs : a.c.ks) + (size_t)id * a.c.Hk)[hk];
  };
  load(h0);
#pragma unroll 1
  for (int hk = h0; hk < h1; ++hk) {
    const T* src = in + hk * st.h;
    unsigned char* dst = (values ? a.c.v : a.c.k) + ((size_t)id * a.c.Hk + hk) * a.c.P * D;
    float* scale = (values ? a.c.vs : a.c.ks) + (size_t)id * a.c.Hk + hk;
    float x[CH][16];
    float amax = 0.f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int e = tid + i * TH, r = r0 + e / C, c = e % C * 16;
      if (r >= r1) continue;
      raw[i].value(x[i]);
      if (turn) {
        float o[16];
        if (chunked) other[i].value(o);
        const float* co = s_cs + (size_t)(r - r0) * rf;
        rotate16(a.rope, src + (t0 + r - p0) * st.t, c, co, s_si + (co - s_cs), o, x[i]);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float m = fabsf(x[i][j]);
        const bool fin = m <= 3.402823466e38f;
        odd |= !fin;
        if (isnan(x[i][j])) x[i][j] = 0.f;
        amax = fmaxf(amax, fin ? m : 0.f);
      }
    }
    if (odd) raise_status(a.status, kDevCheck);
    const float was = had;
    if (hk + 1 < h1) load(hk + 1);
    amax = warp_max(amax);
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TH / 32; ++w) amax = fmaxf(amax, s_max[w]);
    const float need = exp2_int(scale_exponent<F>(amax));
    const bool kept = was > 0.f && was <= 3.402823466e38f;
    const float now = kept ? fmaxf(was, need) : need;
    const float inv = 1.f / now;  // a power of two: exact
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int e = tid + i * TH, r = r0 + e / C, c = e % C;
      if (r >= r1) continue;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = float_to_codes<F>(x[i][4 * j] * inv, x[i][4 * j + 1] * inv, x[i][4 * j + 2] * inv,
                                 x[i][4 * j + 3] * inv);
      *reinterpret_cast<uint4*>(dst + (size_t)r * D + 16 * chunk_place<D>(r, c)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (kept && now != was) {  // the scale grew: earlier tokens are rounded again
      const float f = was * inv;
#pragma unroll 1
      for (int e = tid; e < r0 * C; e += TH) {
        uint4* at = reinterpret_cast<uint4*>(dst + (size_t)e * 16);
        const uint4 old = *at;
        const uint32_t o[4] = {old.x, old.y, old.z, old.w};
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 v = codes_to_float<F>(o[j]);
          w[j] = float_to_codes<F>(v.x * f, v.y * f, v.z * f, v.w * f);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncthreads();  // every thread has read the old scale and the maxima
    if (tid == 0) *scale = now;
  }
}

__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) st4(p + i, make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
}
__device__ __forceinline__ void store16(bf16* p, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// x: 16-code chunks of T rows, y: head, keys or values, z: sequence.
template <typename T, int D, int F>
__global__ void __launch_bounds__(kThreads) read_kernel(CacheIo a) {
  constexpr int C = D / 16;
  pdl_wait();
  const int n = blockIdx.z, hk = blockIdx.y >> 1;
  const bool values = blockIdx.y & 1;
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t j = e / C;
  const int c = (int)(e % C);
  if (j >= a.T) return;
  const int64_t p0 = a.pos[n];
  const int cnt = a.count ? a.count[n] : a.T;
  const bool bad = cnt < 0 || cnt > a.T || (cnt > 0 && (p0 < 0 || !span_ok(a.c, p0, last_of(p0, cnt))));
  if (bad && e == 0) raise_status(a.status, kDevCheck);
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
  if (!bad && j < cnt) {
    const int64_t p = p0 + j;
    const int id = pool_page(a.c, n, (uint32_t)(p >> a.c.log_p));
    if (id < 0) {
      raise_status(a.status, kDevCheck);
    } else {
      const int r = (int)(p & (a.c.P - 1));
      const size_t ph = (size_t)id * a.c.Hk + hk;
      const unsigned char* src = (values ? a.c.v : a.c.k) + (ph * a.c.P + r) * D;
      const float s = (values ? a.c.vs : a.c.ks)[ph];
      const uint4 u = *reinterpret_cast<const uint4*>(src + 16 * chunk_place<D>(r, c));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = codes_to_float<F>(w[i]);
        x[4 * i] = v.x * s, x[4 * i + 1] = v.y * s, x[4 * i + 2] = v.z * s, x[4 * i + 3] = v.w * s;
      }
    }
  }
  const Strides st = values ? a.sv : a.sk;
  T* dst = static_cast<T*>(values ? a.v : a.k) + n * st.n + hk * st.h + j * st.t;
  store16(dst + 16 * c, x);
}

template <typename T, int D, int F, int CH, int TH>
cudaError_t launch_write_as(const CacheIo& a, cudaStream_t s, int* launches) {
  // pages that T tokens touch; a sequence that needs more than its table holds is refused
  const int J = (int)std::min(((int64_t)a.T + a.c.P - 2) / a.c.P + 1, (int64_t)a.c.max_pages);
  const int per = (int64_t)J * a.c.Hk * a.c.N * 2 / kHeads >= ctas_per_wave(4) ? kHeads : 1;
  const dim3 grid(J, 2 * ((a.c.Hk + per - 1) / per), a.c.N);
  const size_t smem = a.rope.turns ? (size_t)min(a.T, a.c.P) * row_floats(a.rope.rot / 2) * 2 * sizeof(float) : 0;
  // The most that any rotation and any count of rows need (a page of 128, all channels), once: near
  // 48 KiB the kernel's own 64 bytes count too, and a limit set per call would be another thread's.
  constexpr int most = 128 * row_floats(D / 2) * 2 * (int)sizeof(float);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = smem ? allow_smem(write_kernel<T, D, F, CH, TH>, most, done) : cudaSuccess;
  if (e != cudaSuccess) return e;
  trace_begin("cache_write", s);
  e = launch_pdl(write_kernel<T, D, F, CH, TH>, grid, dim3(TH), smem, s, a, per);
  trace_end(s);
  ++*launches;
  return e;
}

template <typename T, int D, int F>
cudaError_t launch_write(const CacheIo& a, cudaStream_t s, int* launches) {
  const int chunks = min(a.T, a.c.P) * (D / 16);  // of the new rows of a page, at most
  return chunks <= 32    ? launch_write_as<T, D, F, 1, 32>(a, s, launches)
         : chunks <= 256 ? launch_write_as<T, D, F, 1, 256>(a, s, launches)
         : chunks <= 512 ? launch_write_as<T, D, F, 2, 256>(a, s, launches)
                         : launch_write_as<T, D, F, 2, 512>(a, s, launches);
}

template <typename T, int D, int F>
cudaError_t launch_read(const CacheIo& a, cudaStream_t s, int* launches) {
  const int64_t chunks = (int64_t)a.T * (D / 16);
  const dim3 grid((unsigned)((chunks + kThreads - 1) / kThreads), 2 * a.c.Hk, a.c.N);
  trace_begin("cache_read", s);
  const cudaError_t e = launch_pdl(read_kernel<T, D, F>, grid, dim3(kThreads), 0, s, a);
  trace_end(s);
  ++*launches;
  return e;
}

template <typename T, int D>
cudaError_t by_format(const CacheIo& a, bool write, cudaStream_t s, int* launches) {
  if (a.c.fmt == LIZARD_KV_E4M3)
    return write ? launch_write<T, D, 0>(a, s, launches) : launch_read<T, D, 0>(a, s, launches);
  return write ? launch_write<T, D, 1>(a, s, launches) : launch_read<T, D, 1>(a, s, launches);
}

cudaError_t launch_io(const CacheIo& a, lizard_dtype dt, bool write, cudaStream_t s, int* launches) {
  if (dt == LIZARD_F32)
    return a.c.d == 64 ? by_format<float, 64>(a, write, s, launches)
                       : by_format<float, 128>(a, write, s, launches);
  return a.c.d == 64 ? by_format<bf16, 64>(a, write, s, launches)
                     : by_format<bf16, 128>(a, write, s, launches);
}

}  // namespace

cudaError_t launch_cache_write(const CacheIo& a, lizard_dtype dt, cudaStream_t s, int* launches) {
  return launch_io(a, dt, true, s, launches);
}

cudaError_t launch_cache_read(const CacheIo& a, lizard_dtype dt, cudaStream_t s, int* launches) {
  return launch_io(a, dt, false, s, launches);
}

}  // namespace lz
