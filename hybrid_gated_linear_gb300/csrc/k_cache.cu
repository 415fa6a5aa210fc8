// k_cache.cu -- writing new tokens into the 8-bit paged cache and reading them back.
//
// Write.  One CTA per (sequence, touched page, head, keys or values).  It holds the new
// rows that fall into its page in registers, reduces their largest magnitude, settles the
// page's scale and stores the codes: one pass over the inputs, no second read.  The scale
// is a power of two, so dividing by it is exact, and codes of earlier tokens change only
// when the scale grows (they are then read, rescaled exactly and rounded again).
// Read.  One thread per 16 codes of a row, keys and values in one launch.
#include "kv_cache.cuh"

namespace lz {
namespace {

constexpr int kThreads = 256;

// 16 consecutive elements of a row.
__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 v = ld4(p + i);
    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
  }
}
__device__ __forceinline__ void load16(const bf16* p, float (&x)[16]) {
  const uint4 u0 = *reinterpret_cast<const uint4*>(p), u1 = *reinterpret_cast<const uint4*>(p + 8);
  const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Rotates channels c..c+15 (already in x) of a row; cs holds the row's (cos, sin) pairs.
template <typename T>
__device__ __forceinline__ void rotate16(const RopeArgs& r, const T* row, int c, const float2* cs,
                                         float (&x)[16]) {
  if (c >= r.rot) return;
  if (r.layout == LIZARD_ROPE_INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 2 * i < r.rot) {
        const float2 f = cs[c / 2 + i];
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * f.x - b * f.y;
        x[2 * i + 1] = b * f.x + a * f.y;
      }
    return;
  }
  const int hr = r.rot / 2;
  float o[16];
  if (hr % 16 == 0) {  // the pairs' other channels are a chunk too
    load16(row + (c < hr ? c + hr : c - hr), o);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int e = c + i;
      o[i] = e < r.rot ? ld_f(row + (e < hr ? e + hr : e - hr)) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int e = c + i;
    if (e < r.rot) {
      const bool low = e < hr;
      const float2 f = cs[low ? e : e - hr];
      x[i] = low ? x[i] * f.x - o[i] * f.y : x[i] * f.x + o[i] * f.y;
    }
  }
}

template <typename T, int D, int F, int CH>
__global__ void __launch_bounds__(kThreads) write_kernel(CacheIo a) {
  constexpr int C = D / 16;
  extern __shared__ float2 s_cs[];  // (cos, sin) of every new row's pairs
  __shared__ float s_max[kThreads / 32];
  const int n = blockIdx.z, hk = blockIdx.y >> 1;
  const bool values = blockIdx.y & 1;
  const int tid = threadIdx.x;
  const int64_t p0 = a.pos[n];
  const int cnt = a.count ? a.count[n] : a.T;
  if (cnt == 0) return;
  const bool bad = cnt < 0 || cnt > a.T || p0 < 0 || !span_ok(a.c, p0, p0 + cnt - 1);
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
  const T* src = static_cast<const T*>(values ? a.v : a.k) + n * st.n + hk * st.h;
  unsigned char* dst = (values ? a.c.v : a.c.k) + ((size_t)id * a.c.Hk + hk) * a.c.P * D;
  float* scale = (values ? a.c.vs : a.c.ks) + (size_t)id * a.c.Hk + hk;
  const bool turn = !values && a.rope.turns;
  const int pairs = a.rope.rot / 2;
  if (turn) {
    for (int e = tid; e < (r1 - r0) * pairs; e += kThreads) {
      const int r = e / pairs, i = e - r * pairs;
      float2 f;
      rope_angle(a.rope.turns[i], t0 + r0 + r, a.rope.factor, f.x, f.y);
      s_cs[e] = f;
    }
    __syncthreads();
  }

  float x[CH][16];
  float amax = 0.f;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int e = tid + i * kThreads, r = e / C, c = e % C * 16;
    if (r < r0 || r >= r1) continue;
    const T* row = src + (t0 + r - p0) * st.t;
    load16(row + c, x[i]);
    if (turn) rotate16(a.rope, row, c, s_cs + (r - r0) * pairs, x[i]);
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
  amax = warp_max(amax);
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  const float had = r0 > 0 ? *scale : 0.f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  const float need = exp2_int(scale_exponent<F>(amax));
  const bool kept = had > 0.f && had <= 3.402823466e38f;
  const float now = kept ? fmaxf(had, need) : need;
  const float inv = 1.f / now;  // a power of two: exact
  const bool grew = kept && now != had;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int e = tid + i * kThreads, r = e / C, c = e % C;
    uint4* at = reinterpret_cast<uint4*>(dst + (size_t)r * D + 16 * chunk_place<D>(r, c));
    if (r >= r0 && r < r1) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = float_to_codes<F>(x[i][4 * j] * inv, x[i][4 * j + 1] * inv, x[i][4 * j + 2] * inv,
                                 x[i][4 * j + 3] * inv);
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (r < r0 && grew) {
      const float f = had * inv;
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
  // every thread has read the old scale before the barrier above
  if (tid == 0) *scale = now;
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
  const int n = blockIdx.z, hk = blockIdx.y >> 1;
  const bool values = blockIdx.y & 1;
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t j = e / C;
  const int c = (int)(e % C);
  if (j >= a.T) return;
  const int64_t p0 = a.pos[n];
  const int cnt = a.count ? a.count[n] : a.T;
  const bool bad = cnt < 0 || cnt > a.T || (cnt > 0 && (p0 < 0 || !span_ok(a.c, p0, p0 + cnt - 1)));
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

template <typename T, int D, int F, int CH>
cudaError_t launch_write_ch(const CacheIo& a, cudaStream_t s, int* launches) {
  const dim3 grid((a.T + a.c.P - 2) / a.c.P + 1, 2 * a.c.Hk, a.c.N);
  const size_t smem = (size_t)min(a.T, a.c.P) * (a.rope.rot / 2) * sizeof(float2);
  cudaError_t e = cudaFuncSetAttribute(write_kernel<T, D, F, CH>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * (D / 2) * 8);
  if (e != cudaSuccess) return e;
  trace_begin("cache_write", s);
  write_kernel<T, D, F, CH><<<grid, kThreads, smem, s>>>(a);
  trace_end(s);
  ++*launches;
  return cudaGetLastError();
}

template <typename T, int D, int F>
cudaError_t launch_write(const CacheIo& a, cudaStream_t s, int* launches) {
  const int ch = a.c.P * (D / 16) / kThreads;  // 16-code chunks per thread
  return ch >= 4   ? launch_write_ch<T, D, F, 4>(a, s, launches)
         : ch == 2 ? launch_write_ch<T, D, F, 2>(a, s, launches)
                   : launch_write_ch<T, D, F, 1>(a, s, launches);
}

template <typename T, int D, int F>
cudaError_t launch_read(const CacheIo& a, cudaStream_t s, int* launches) {
  const int64_t chunks = (int64_t)a.T * (D / 16);
  const dim3 grid((unsigned)((chunks + kThreads - 1) / kThreads), 2 * a.c.Hk, a.c.N);
  trace_begin("cache_read", s);
  read_kernel<T, D, F><<<grid, kThreads, 0, s>>>(a);
  trace_end(s);
  ++*launches;
  return cudaGetLastError();
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
