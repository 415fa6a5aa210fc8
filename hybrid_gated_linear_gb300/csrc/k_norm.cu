// k_norm.cu -- layer norm of rows of d channels and its backward.
//   n = (x - mean) r,  r = 1 / sqrt(mean((x - mean)^2) + eps),  y = n w + b
//   a = dy w,  dx = r (a - mean(a) - n mean(a n)),  dw = sum dy n,  db = sum dy
// Both are bound by memory (x in, y out; x and dy in, dx out).  A row lies in the registers of
// TPR threads, 16 channels each, from its one read to its one write: the mean is summed first, the
// variance around it second, both from registers, so that a large mean costs no digits and the
// backward needs nothing but x.  Forward, 2 x 32 x 4096 rows of 128 in bf16: 27 us, 5.0 TB/s, 75% of the copy
// rate (the arithmetic of a row and its start); backward 35 us, 85%; 8191 rows of 4096 backward 47 us, 63%
// (two turns of sums over eight warps a row).  There arithmetic on pairs and row indices by addition made it
// 72 -> 55 us, two turns of sums instead of three 54.6, one round of blocks 47.
#include "lizard_dev.cuh"
#include "lizard_internal.h"

namespace lz {
namespace {

constexpr int kEpt = 16;  // channels of a thread
constexpr int kBlock = 256;

template <typename T>
struct Frag {
  static constexpr int V = 16 / (int)sizeof(T);  // channels of a 16-byte vector
  static constexpr int NV = kEpt / V;
  uint4 v[NV];
};

// A thread's channels in pairs, for the instructions that take two.
constexpr int kP = kEpt / 2;
__device__ __forceinline__ void unpack(const Frag<float>& f, float2 (&o)[kP]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = make_float2(__uint_as_float(f.v[i].x), __uint_as_float(f.v[i].y));
    o[2 * i + 1] = make_float2(__uint_as_float(f.v[i].z), __uint_as_float(f.v[i].w));
  }
}
__device__ __forceinline__ void unpack(const Frag<bf16>& f, float2 (&o)[kP]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {f.v[i].x, f.v[i].y, f.v[i].z, f.v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) o[4 * i + j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
  }
}
__device__ __forceinline__ void pack(const float2 (&o)[kP], Frag<float>& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f.v[i] = make_uint4(__float_as_uint(o[2 * i].x), __float_as_uint(o[2 * i].y), __float_as_uint(o[2 * i + 1].x),
                        __float_as_uint(o[2 * i + 1].y));
}
__device__ __forceinline__ void pack(const float2 (&o)[kP], Frag<bf16>& f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(o[4 * i + j].x, o[4 * i + j].y);
      w[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
    f.v[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Thread `lane` of a row holds the vectors lane, lane + TPR, ...; those past the row are zeros.
template <typename T, int TPR>
__device__ __forceinline__ void load(const T* row, int lane, int d, Frag<T>& f) {
#pragma unroll
  for (int i = 0; i < Frag<T>::NV; ++i) {
    const int c = (lane + TPR * i) * Frag<T>::V;
    f.v[i] = row && c < d ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
  }
}
template <typename T, int TPR>
__device__ __forceinline__ void store(T* row, int lane, int d, const Frag<T>& f) {
#pragma unroll
  for (int i = 0; i < Frag<T>::NV; ++i) {
    const int c = (lane + TPR * i) * Frag<T>::V;
    if (c < d) *reinterpret_cast<uint4*>(row + c) = f.v[i];
  }
}
// Whether the thread's element e lies inside the row.
template <typename T, int TPR>
__device__ __forceinline__ bool inside(int lane, int d, int e) {
  return (lane + TPR * (e / Frag<T>::V)) * Frag<T>::V < d;
}

// Sums over the TPR threads of a row, the same in all of them.  Rows of more than a warp use
// `part` and a barrier: every thread of the block calls, and two calls in turn use `part` of two
// parities, so that the second's writes do not meet the first's reads.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* part, int parity) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  if (TPR > 32) {
    constexpr int W = TPR > 32 ? TPR / 32 : 1;  // warps of a row
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float* p = part + parity * 64;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) p[warp * 2 + k] = s[k];
    __syncthreads();
    const int w0 = warp / W * W;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float t = lane < W ? p[(w0 + lane) * 2 + k] : 0.f;
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      s[k] = W < 32 ? __shfl_sync(0xffffffffu, t, 0) : t;
    }
  }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// x becomes x - mean; returns 1 / sqrt(var + eps).
template <typename T, int TPR>
__device__ __forceinline__ float centre(float2 (&x)[kP], int lane, int d, float eps, float inv_d, float* part) {
  float2 t = x[0];
#pragma unroll
  for (int e = 1; e < kP; ++e) t = f2_add(t, x[e]);
  float s[1] = {t.x + t.y};
  row_sum<TPR>(s, part, 0);
  const float2 minus = both(-s[0] * inv_d);
  t = both(0.f);
#pragma unroll
  for (int e = 0; e < kP; ++e) {
    x[e] = inside<T, TPR>(lane, d, 2 * e) ? f2_add(x[e], minus) : both(0.f);
    t = f2_fma(x[e], x[e], t);
  }
  s[0] = t.x + t.y;
  row_sum<TPR>(s, part, 1);
  return rsqrtf(fmaf(s[0], inv_d, eps));
}

// Row r (of rows of all heads, or of one head) as n, h, t; the axis with the smaller stride of x
// is the inner one, so that neighbouring threads' rows are neighbours in memory.
struct Index {
  uint32_t n, h, t;
};
__device__ __forceinline__ Index index_of(const NormCall& a, uint32_t r, bool heads_inner) {
  Index i;
  if (heads_inner) {
    const uint32_t q = r / a.H;
    i.h = r - q * a.H;
    i.n = q / a.T;
    i.t = q - i.n * a.T;
  } else {
    const uint32_t q = r / a.T;
    i.t = r - q * a.T;
    i.n = q / a.H;
    i.h = q - i.n * a.H;
  }
  return i;
}
// The index `step` rows on, by its parts (a division costs what a third of a row's arithmetic does).
struct Walk {
  uint32_t in, mid, out;  // the inner axis, the next, and n
  __device__ __forceinline__ void start(uint32_t r, uint32_t n_in, uint32_t n_mid) {
    const uint32_t q = r / n_in;
    in = r - q * n_in, out = q / n_mid, mid = q - out * n_mid;
  }
  __device__ __forceinline__ void advance(const Walk& step, uint32_t n_in, uint32_t n_mid) {
    in += step.in, mid += step.mid, out += step.out;
    if (in >= n_in) in -= n_in, ++mid;
    if (mid >= n_mid) mid -= n_mid, ++out;
  }
};
__device__ __forceinline__ int64_t offset(const Strides& s, const Index& i) {
  return i.n * s.n + i.h * s.h + i.t * s.t;
}

template <typename T, int TPR>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock) norm_fwd_kernel(NormCall a, uint32_t rows, bool heads_inner) {
  constexpr int RPB = (TPR > kBlock ? TPR : kBlock) / TPR;
  __shared__ float part[128];
  pdl_wait();
  const int lane = threadIdx.x % TPR;
  const uint32_t r = blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = r < rows;
  const Index i = index_of(a, live ? r : 0, heads_inner);
  Frag<T> f, fw, fb;
  load<T, TPR>(live ? static_cast<const T*>(a.x) + offset(a.sx, i) : nullptr, lane, a.d, f);
  const int64_t wo = a.per_head ? (int64_t)i.h * a.d : 0;
  load<T, TPR>(a.w ? static_cast<const T*>(a.w) + wo : nullptr, lane, a.d, fw);
  load<T, TPR>(a.b ? static_cast<const T*>(a.b) + wo : nullptr, lane, a.d, fb);
  float2 x[kP], w[kP], b[kP];
  unpack(f, x);
  const float2 rs = both(centre<T, TPR>(x, lane, a.d, a.eps, 1.f / a.d, part));
  unpack(fw, w);
  unpack(fb, b);
#pragma unroll
  for (int e = 0; e < kP; ++e) x[e] = f2_fma(f2_mul(x[e], rs), a.w ? w[e] : both(1.f), b[e]);
  pack(x, f);
  if (live) store<T, TPR>(static_cast<T*>(a.y) + offset(a.sy, i), lane, a.d, f);
}

// Rows on their way to a thread of the backward: a ring of its own vectors of x and dy in shared memory,
// filled by asynchronous copies: memory's latency times its rate is about 40 KB for each SM, a row ahead in
// registers 32 (2 x 32 x 4096 rows of 128: 49 us that way, 43 this).
template <typename T, int THREADS>
struct Ring {
  static constexpr int NV = Frag<T>::NV, kStage = 2 * NV * THREADS * 16;
  static constexpr int D = kStage <= 16384 ? 4 : kStage <= 65536 ? 3 : 1;
  static constexpr int kBytes = D * kStage;
};
__device__ __forceinline__ void copy16(uint4* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(there ? 16 : 0)
               : "memory");
}

// Block (x, y): every gridDim.x-th group of rows of head y (per_head) or of all rows.  The sums of
// dw and db stay in the threads' registers until the block's last row; then the block's rows are
// added up in a fixed order into part[y][x][2][d].
template <typename T, int TPR>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock) norm_bwd_kernel(NormCall a, uint32_t rows, bool heads_inner) {
  constexpr int THREADS = TPR > kBlock ? TPR : kBlock, RPB = THREADS / TPR;
  using R = Ring<T, THREADS>;
  // the ring; after the last row in its place [warps][2][d] sums for rows within a warp, [RPB][2][d] for wider ones
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float part[128];
  pdl_wait();
  const int lane = threadIdx.x % TPR;
  const T* xs = static_cast<const T*>(a.x);
  const T* dys = static_cast<const T*>(a.dy);
  // rows of one head: tokens of sequences; of all heads: in the order of index_of
  const uint32_t n_in = a.per_head || !heads_inner ? a.T : a.H, n_mid = a.per_head ? 1 : heads_inner ? a.T : a.H;
  auto at = [&](const Walk& p) {
    if (a.per_head) return Index{p.out, blockIdx.y, p.in};
    return heads_inner ? Index{p.out, p.in, p.mid} : Index{p.out, p.mid, p.in};
  };
  float2 w[kP], dw[kP], db[kP];
  {
    Frag<T> f;
    load<T, TPR>(a.w ? static_cast<const T*>(a.w) + (a.per_head ? (int64_t)blockIdx.y * a.d : 0) : nullptr, lane, a.d, f);
    unpack(f, w);
  }
#pragma unroll
  for (int e = 0; e < kP; ++e) {
    if (!a.w) w[e] = both(1.f);
    dw[e] = db[e] = both(0.f);
  }
  const float inv_d = 1.f / a.d;
  const uint32_t step = gridDim.x * RPB, first = blockIdx.x * RPB, own = first + threadIdx.x / TPR;
  Walk next, here, by;  // of the row to fetch, of the row at work, of a step
  next.start(own, n_in, n_mid);
  here = next;
  by.start(step, n_in, n_mid);
  auto fetch = [&](uint32_t r, int stage) {  // (one group a row, there or not)
    if (r < rows) {
      const Index i = at(next);
      const T *px = xs + offset(a.sx, i), *py = dys + offset(a.sdy, i);
      uint4* d = ring + stage * (2 * R::NV * THREADS) + threadIdx.x;
#pragma unroll
      for (int k = 0; k < R::NV; ++k) {
        const int c = (lane + TPR * k) * Frag<T>::V;
        const bool there = c < a.d;
        copy16(d + k * THREADS, px + (there ? c : 0), there);
        copy16(d + (R::NV + k) * THREADS, py + (there ? c : 0), there);
      }
    }
    next.advance(by, n_in, n_mid);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int k = 0; k < R::D; ++k) fetch(own + k * step, k);
  int stage = 0;
  for (uint32_t base = first; base < rows; base += step) {
    const uint32_t r = own + (base - first);
    float2 x[kP], dy[kP];
    Frag<T> f, g;
    asm volatile("cp.async.wait_group %0;" ::"n"(R::D - 1) : "memory");
    const uint4* d = ring + stage * (2 * R::NV * THREADS) + threadIdx.x;
    const bool live = r < rows;
#pragma unroll
    for (int k = 0; k < R::NV; ++k) {
      f.v[k] = live ? d[k * THREADS] : make_uint4(0, 0, 0, 0);
      g.v[k] = live ? d[(R::NV + k) * THREADS] : make_uint4(0, 0, 0, 0);
    }
    unpack(f, x);
    unpack(g, dy);
    fetch(r + R::D * step, stage);  // (below 2^32: rows are below 2^31, a step below 2^16)
    stage = stage + 1 == R::D ? 0 : stage + 1;
    // two sums in one turn: of x and a, then, around the mean, of x^2 and a x
    float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      s0 = f2_add(s0, x[e]);
      s1 = f2_fma(dy[e], w[e], s1);
    }
    float s[2] = {s0.x + s0.y, s1.x + s1.y};
    row_sum<TPR>(s, part, 0);
    const float2 minus = both(-s[0] * inv_d), m0 = both(-s[1] * inv_d);
    s0 = s1 = both(0.f);
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      x[e] = inside<T, TPR>(lane, a.d, 2 * e) ? f2_add(x[e], minus) : both(0.f);
      s0 = f2_fma(x[e], x[e], s0);
      s1 = f2_fma(f2_mul(dy[e], w[e]), x[e], s1);
    }
    s[0] = s0.x + s0.y, s[1] = s1.x + s1.y;
    row_sum<TPR>(s, part, 1);
    const float r1 = rsqrtf(fmaf(s[0], inv_d, a.eps));
    const float2 rs = both(r1), m1 = both(-s[1] * r1 * inv_d);
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      x[e] = f2_mul(x[e], rs);
      db[e] = f2_add(db[e], dy[e]);
      dw[e] = f2_fma(dy[e], x[e], dw[e]);
      x[e] = f2_mul(rs, f2_fma(x[e], m1, f2_fma(dy[e], w[e], m0)));
    }
    Frag<T> o;
    pack(x, o);
    if (live && a.y) store<T, TPR>(static_cast<T*>(a.y) + offset(a.sy, at(here)), lane, a.d, o);
    here.advance(by, n_in, n_mid);
  }
  if (!a.part) return;
  // every copy that was started has been waited for by its row, but not by the other threads of the block
  float* sums = reinterpret_cast<float*>(ring);
  __syncthreads();
  // rows of one warp, then the block's warps (or rows) one after the other
  constexpr int PARTS = TPR < 32 ? THREADS / 32 : RPB;
#pragma unroll
  for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      dw[e].x += __shfl_xor_sync(0xffffffffu, dw[e].x, o), dw[e].y += __shfl_xor_sync(0xffffffffu, dw[e].y, o);
      db[e].x += __shfl_xor_sync(0xffffffffu, db[e].x, o), db[e].y += __shfl_xor_sync(0xffffffffu, db[e].y, o);
    }
  float* mine = PARTS == 1 ? a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.d
                           : sums + (TPR < 32 ? threadIdx.x / 32 : threadIdx.x / TPR) * 2 * a.d;
  if (TPR >= 32 || threadIdx.x % 32 < TPR) {
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      const int c = (lane + TPR * (2 * e / Frag<T>::V)) * Frag<T>::V + 2 * e % Frag<T>::V;
      if (inside<T, TPR>(lane, a.d, 2 * e)) {
        *reinterpret_cast<float2*>(mine + c) = dw[e];
        *reinterpret_cast<float2*>(mine + a.d + c) = db[e];
      }
    }
  }
  if (PARTS == 1) return;
  __syncthreads();
  float* out = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.d;
  for (int c = threadIdx.x; c < 2 * a.d; c += THREADS) {
    float s = 0.f;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) s += sums[p * 2 * a.d + c];
    out[c] = s;
  }
}

// dw, db from the blocks' parts [sets][parts][2][d]: 32 columns and 32 strands of parts a block,
// the strands joined in order.
__global__ void __launch_bounds__(1024) norm_weights_kernel(const float* part, int parts, int d, float* dw, float* db) {
  __shared__ float s[32][33];
  pdl_wait();
  const int c = blockIdx.x * 32 + threadIdx.x;
  const float* p = part + (int64_t)blockIdx.y * parts * 2 * d + c;
  float sum = 0.f;
  if (c < 2 * d) {
#pragma unroll 8
    for (int k = threadIdx.y; k < parts; k += 32) sum += p[(int64_t)k * 2 * d];
  }
  s[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y || c >= 2 * d) return;
  sum = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) sum += s[k][threadIdx.x];
  float* o = c < d ? dw : db;
  if (o) o[(int64_t)blockIdx.y * d + (c < d ? c : c - d)] = sum;
}

// Threads of a row: 16 channels each, a power of two from 4 on.
int threads_per_row(int d) {
  int t = 4;
  while (t * kEpt < d) t *= 2;
  return t;
}
int rows_per_block(int d) {
  const int t = threads_per_row(d);
  return t >= kBlock ? 1 : kBlock / t;
}
// Blocks that share the rows of one set of weights in the backward: one round of the blocks that SMs
// hold, over all sets; a second round costs more than it fills (bf16, two rounds, then one: 32 heads' rows of
// 128 36.1 / 33.3 us, 8191 rows of 4096 55.0 / 47.3, 4096 rows of 8192 62 / 54).  An SM holds two blocks of 256
// threads, by their registers and by their rings (the sums of the block's rows lie in the ring's place; behind
// it, in fp32, a block had the SM to itself and half of the blocks came second: 61680 rows of 544 93 us, 75
// this way).  But one fp32 ring of 96 KB is what keeps memory busy, and a second one in its way where rows
// fill it: 134 MB of rows of 1024, 2048, 4096 two blocks 72, 73, 75 us, one 66, 64, 66; of 1792 75 / 66, of
// 1536 70 / 73, of 1280 67 / 83; to 512 channels the same within 3.  (152 SMs: written down, so that the
// workspace does not ask for a device.)
int bwd_blocks(int64_t rows, int sets, int d, bool f32) {
  const int64_t most = (rows + rows_per_block(d) - 1) / rows_per_block(d);
  const int t = threads_per_row(d);
  const int per_sm = t > kBlock || (f32 && sets == 1 && t > 32 && 4 * d > 3 * t * kEpt) ? 1 : 2;
  int64_t n = (int64_t)152 * per_sm / sets;
  n = n < most ? n : most;
  return (int)(n < 1 ? 1 : n);
}
bool heads_inner(const NormCall& a) { return a.H > 1 && (a.T == 1 || a.sx.h < a.sx.t); }

template <typename T, int TPR>
cudaError_t fwd(const NormCall& a, cudaStream_t s) {
  const uint32_t rows = (uint32_t)a.N * a.H * a.T;
  const int rpb = rows_per_block(a.d);
  return launch_pdl(norm_fwd_kernel<T, TPR>, dim3((rows + rpb - 1) / rpb), dim3(TPR > kBlock ? TPR : kBlock), 0, s, a,
                    rows, heads_inner(a));
}
template <typename T, int TPR>
cudaError_t bwd(const NormCall& a, cudaStream_t s) {
  const uint32_t rows = (uint32_t)a.N * a.T * (a.per_head ? 1 : a.H);
  const int sets = a.per_head ? a.H : 1;
  constexpr int threads = TPR > kBlock ? TPR : kBlock;
  static std::atomic<uint64_t> done{0};
  static_assert(Ring<T, threads>::kBytes >= 32768, "the sums of a block's rows lie in the ring's place");
  const cudaError_t e = allow_smem(norm_bwd_kernel<T, TPR>, Ring<T, threads>::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_bwd_kernel<T, TPR>, dim3(bwd_blocks(rows, sets, a.d, sizeof(T) == 4), sets), dim3(threads),
                    Ring<T, threads>::kBytes, s, a, rows, heads_inner(a));
}

template <typename T>
cudaError_t dispatch(const NormCall& a, bool back, cudaStream_t s) {
  switch (threads_per_row(a.d)) {
#define LZ_NORM(n) \
  case n: return back ? bwd<T, n>(a, s) : fwd<T, n>(a, s);
    LZ_NORM(4) LZ_NORM(8) LZ_NORM(16) LZ_NORM(32) LZ_NORM(64) LZ_NORM(128) LZ_NORM(256) LZ_NORM(512) LZ_NORM(1024)
#undef LZ_NORM
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t norm_part_floats(int N, int H, int T, int d, bool per_head, lizard_dtype dt) {
  const int sets = per_head ? H : 1;
  return (size_t)sets * bwd_blocks((int64_t)N * T * (per_head ? 1 : H), sets, d, dt == LIZARD_F32) * 2 * d;
}

cudaError_t launch_norm_fwd(const NormCall& a, lizard_dtype dt, cudaStream_t s, int* launches) {
  trace_begin("norm_fwd", s);
  const cudaError_t e = dt == LIZARD_F32 ? dispatch<float>(a, false, s) : dispatch<bf16>(a, false, s);
  trace_end(s);
  ++*launches;
  return e;
}

cudaError_t launch_norm_bwd(const NormCall& a, lizard_dtype dt, cudaStream_t s, int* launches) {
  trace_begin("norm_bwd", s);
  cudaError_t e = dt == LIZARD_F32 ? dispatch<float>(a, true, s) : dispatch<bf16>(a, true, s);
  trace_end(s);
  ++*launches;
  if (e != cudaSuccess || !a.part) return e;
  const int sets = a.per_head ? a.H : 1;
  const int parts = bwd_blocks((int64_t)a.N * a.T * (a.per_head ? 1 : a.H), sets, a.d, dt == LIZARD_F32);
  trace_begin("norm_weights", s);
  e = launch_pdl(norm_weights_kernel, dim3((2 * a.d + 31) / 32, sets), dim3(32, 32), 0, s,
                 static_cast<const float*>(a.part), parts, a.d, a.dw, a.db);
  trace_end(s);
  ++*launches;
  return e;
}

}  // namespace lz
