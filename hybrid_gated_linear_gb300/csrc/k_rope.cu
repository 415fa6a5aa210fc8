// k_rope.cu -- rotary positions of queries and keys in one launch, forward and adjoint.
//
// Pair i < rot/2 of every head of a token at position p is turned by p theta_i (include/
// lizard.h states the layouts and scalings); the adjoint turns by -p theta_i, so both are
// this kernel with the sign of the sine changed.  Two loads and two stores of a row per
// head and a handful of FMAs per pair: memory bound, so each thread computes the cosines
// and sines of its VP pairs once, in registers, and walks over the heads of its token with
// 16-byte accesses.  Heads are shared out over several threads where tokens are few.
// Measured: bf16, 8 x 2048 tokens x 64 heads of 128, token-major: 92 us, 5.8 TB/s (86% of the
// measured copy rate); fp32, 2 x 1999 tokens x 30 heads: 20 us.
#include "kv_cache.cuh"

namespace lz {
namespace {

constexpr int kThreads = 256;

// VP consecutive elements, aligned to their size together, in one access of up to 16 bytes.
template <int BYTES> struct Word;
template <> struct Word<2> { typedef unsigned short type; };
template <> struct Word<4> { typedef uint32_t type; };
template <> struct Word<8> { typedef uint2 type; };
template <> struct Word<16> { typedef uint4 type; };
template <typename T, int VP>
union Packed {
  typename Word<VP * sizeof(T)>::type word;
  T v[VP];
  __device__ __forceinline__ Packed() {}
};
template <typename T, int VP>
__device__ __forceinline__ void load_v(const T* p, float (&x)[VP]) {
  Packed<T, VP> u;
  u.word = *reinterpret_cast<const decltype(u.word)*>(p);
#pragma unroll
  for (int i = 0; i < VP; ++i) x[i] = ld_f(&u.v[i]);
}
template <typename T, int VP>
__device__ __forceinline__ void store_v(T* p, const float (&x)[VP]) {
  Packed<T, VP> u;
#pragma unroll
  for (int i = 0; i < VP; ++i) u.v[i] = cvt_out<T>(x[i]);
  *reinterpret_cast<decltype(u.word)*>(p) = u.word;
}

// One thread per (token, unit of 2 VP channels, group of `hpt` heads).  The first units hold VP
// pairs each and are rotated (neighbours that are pairs may end inside a unit); the others are
// copied.  VP = 16 bytes' worth of elements, fewer where the halves' distance rot / 2 is not a
// multiple of that (11 x 752 tokens x 26 heads of 64, rot = 56, bf16: 31 us with single elements,
// 12 with these; an odd number of pairs in halves is left with those).
template <typename T, int VP>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeCall a, int units, int hpt,
                                                        int groups) {
  pdl_wait();
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t total = (int64_t)a.N * a.T * units * groups;
  if (idx >= total) return;
  const int u = (int)(idx % units);
  const int64_t r = idx / units;
  const int64_t nt = r % ((int64_t)a.N * a.T);
  const int g = (int)(r / ((int64_t)a.N * a.T));
  const int n = (int)(nt / a.T), t = (int)(nt % a.T);
  const int pairs = a.rope.rot / 2;
  const bool turned = u * VP < pairs;
  const bool half = a.rope.layout == LIZARD_ROPE_HALF;
  // channels of the unit's two vectors
  const int c0 = turned && half ? u * VP : u * 2 * VP;
  const int c1 = turned && half ? c0 + a.rope.rot / 2 : c0 + VP;
  float co[VP], si[VP];
  if (turned) {
    const int64_t p = a.positions ? a.positions[nt] : t;
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      rope_angle(a.rope.turns[min(u * VP + i, pairs - 1)], p, a.rope.factor, co[i], si[i]);
      si[i] *= a.sign;
    }
  }
  const int h1 = min(a.H + a.Hk, (g + 1) * hpt);
#pragma unroll 2
  for (int h = g * hpt; h < h1; ++h) {
    const bool q = h < a.H;
    const int hh = q ? h : h - a.H;
    const Strides& sx = q ? a.sxq : a.sxk;
    const Strides& sy = q ? a.syq : a.syk;
    const T* x = static_cast<const T*>(q ? a.xq : a.xk) + n * sx.n + hh * sx.h + t * sx.t;
    T* y = static_cast<T*>(q ? a.yq : a.yk) + n * sy.n + hh * sy.h + t * sy.t;
    float v[VP], w[VP];
    load_v<T, VP>(x + c0, v);
    load_v<T, VP>(x + c1, w);
    if (turned && half) {
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        const float p = v[i], s = w[i];
        v[i] = p * co[i] - s * si[i];
        w[i] = s * co[i] + p * si[i];
      }
    } else if (VP > 1 && turned) {
      // neighbours are pairs (VP > 1 always): pairs 0..VP/2-1 lie in v, the others in w
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        float* e = i < VP / 2 ? &v[2 * i] : &w[(2 * i - VP) & (VP - 1)];
        const float p = e[0], s = e[VP > 1];
        if (u * VP + i < pairs) {
          e[0] = p * co[i] - s * si[i];
          e[VP > 1] = s * co[i] + p * si[i];
        }
      }
    }
    store_v<T, VP>(y + c0, v);
    store_v<T, VP>(y + c1, w);
  }
}

template <typename T, int VP>
cudaError_t launch(const RopeCall& a, cudaStream_t s, int* launches) {
  const int units = a.d / (2 * VP), heads = a.H + a.Hk;
  const int64_t lanes = (int64_t)a.N * a.T * units;
  const int64_t want = (int64_t)ctas_per_wave(4) * kThreads;
  int64_t hpt = lanes * heads / want;
  hpt = hpt < 1 ? 1 : hpt > heads ? heads : hpt;
  const int groups = (int)((heads + hpt - 1) / hpt);
  const int64_t blocks = (lanes * groups + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  trace_begin("rope", s);
  const cudaError_t e = launch_pdl(rope_kernel<T, VP>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, units,
                                   (int)hpt, groups);
  trace_end(s);
  ++*launches;
  return e;
}

template <typename T>
cudaError_t launch_typed(const RopeCall& a, cudaStream_t s, int* launches) {
  constexpr int V = 16 / sizeof(T);
  const int pairs = a.rope.layout == LIZARD_ROPE_HALF ? a.rope.rot / 2 : V;
  if (pairs % V == 0 && a.d % (2 * V) == 0) return launch<T, V>(a, s, launches);
  if (sizeof(T) == 2 && pairs % 4 == 0) return launch<T, 4>(a, s, launches);
  return pairs % 2 == 0 ? launch<T, 2>(a, s, launches) : launch<T, 1>(a, s, launches);
}

}  // namespace

cudaError_t launch_rope(const RopeCall& a, lizard_dtype dt, cudaStream_t s, int* launches) {
  return dt == LIZARD_F32 ? launch_typed<float>(a, s, launches) : launch_typed<bf16>(a, s, launches);
}

}  // namespace lz
