// k_decay_step.cu -- the recurrent form of the linear attention with a decay per head:
//   h <- g h + k v^T,  y = scale q^T h,  one token after the other.
// Memory bound: a state of dk dv fp32 is read and written once for 4 dk dv operations a token.  A CTA
// takes DVS of the dv columns of one head's state, which no other CTA needs for its columns of y, and
// holds them in registers over the call's tokens: thread (r, c) has rows r, r + R, ... of 4 columns.
// 64 sequences x 32 heads of 128 x 128: 42 us, 6.4 TB/s, 94% of the copy rate.
// y is summed over a thread's rows, then over the R row strands through shared memory.
#include "lizard_dev.cuh"
#include "lizard_internal.h"

namespace lz {
namespace {

constexpr int kThreads = 256;

template <typename T, int DK, int DVS>
__global__ void __launch_bounds__(kThreads) decay_step_kernel(DecayStep a) {
  constexpr int C = DVS / 4, R = kThreads / C, NR = DK / R;  // column quads, row strands, rows of a thread
  static_assert(NR >= 1 && R * NR == DK, "rows of the state divide among the strands");
  __shared__ float sq[DK], sk[DK];
  __shared__ __align__(16) float ys[kThreads / 32][DVS];
  pdl_wait();
  const int slices = a.dv / DVS;
  const int unit = blockIdx.x / slices, c0 = (blockIdx.x - unit * slices) * DVS;
  const int n = unit / a.H, h = unit - n * a.H, hk = h / a.G;
  const int tid = threadIdx.x, c = tid % C, r = tid / C;
  const int64_t at = ((int64_t)unit * DK + r) * a.dv + c0 + 4 * c;
  float4 s[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i)
    s[i] = a.h_in ? *reinterpret_cast<const float4*>(a.h_in + at + (int64_t)i * R * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
  int count = a.L;
  if (a.count) {
    count = a.count[n];
    if (count < 0 || count > a.L) {
      if (tid == 0) raise_status(a.status, kDevCheck);
      count = 0;
    }
  }
  const T* q = static_cast<const T*>(a.q) + n * a.sq.n + h * a.sq.h;
  const T* k = static_cast<const T*>(a.k) + n * a.sk.n + hk * a.sk.h;
  const T* v = static_cast<const T*>(a.v) + n * a.sv.n + hk * a.sv.h + c0 + 4 * c;
  const float* lg = a.lg + n * a.sg.n + h * a.sg.h;
  T* y = static_cast<T*>(a.y) + n * a.sy.n + h * a.sy.h + c0;
  for (int t = 0; t < count; ++t) {
    if (tid < DK) sq[tid] = ld_f(q + t * a.sq.t + tid) * a.scale;
    if (tid >= kThreads - DK) sk[tid - (kThreads - DK)] = ld_f(k + t * a.sk.t + tid - (kThreads - DK));
    const float4 vt = ld4(v + t * a.sv.t);
    const float g = expf(lg[t * a.sg.t]);
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float kr = sk[r + i * R], qr = sq[r + i * R];
      // a decay of 0 leaves nothing, whatever the state was
      s[i].x = fmaf(kr, vt.x, g == 0.f ? 0.f : g * s[i].x);
      s[i].y = fmaf(kr, vt.y, g == 0.f ? 0.f : g * s[i].y);
      s[i].z = fmaf(kr, vt.z, g == 0.f ? 0.f : g * s[i].z);
      s[i].w = fmaf(kr, vt.w, g == 0.f ? 0.f : g * s[i].w);
      o.x = fmaf(qr, s[i].x, o.x);
      o.y = fmaf(qr, s[i].y, o.y);
      o.z = fmaf(qr, s[i].z, o.z);
      o.w = fmaf(qr, s[i].w, o.w);
    }
#pragma unroll
    for (int x = C; x < 32; x <<= 1) {  // the row strands of a warp
      o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
    }
    if (tid % 32 < C) *reinterpret_cast<float4*>(&ys[tid / 32][4 * c]) = o;
    __syncthreads();
    if (tid < DVS) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) sum += ys[w][tid];
      y[t * a.sy.t + tid] = cvt_out<T>(sum);
    }
  }
  for (int t = count; t < a.L; ++t)
    if (tid < DVS) y[t * a.sy.t + tid] = cvt_out<T>(0.f);
  if (!a.h_out) return;
#pragma unroll
  for (int i = 0; i < NR; ++i) *reinterpret_cast<float4*>(a.h_out + at + (int64_t)i * R * a.dv) = s[i];
}

template <typename T, int DK, int DVS>
cudaError_t launch(const DecayStep& a, cudaStream_t s) {
  const int64_t blocks = (int64_t)a.B * a.H * (a.dv / DVS);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_pdl(decay_step_kernel<T, DK, DVS>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
}

template <typename T, int DK>
cudaError_t dispatch(const DecayStep& a, cudaStream_t s) {
  // whole rows (the longest runs of memory) where they fill the GPU, else the columns are split
  const int64_t units = (int64_t)a.B * a.H, want = ctas_per_wave(2);
  if (a.dv == 128 && units >= want) return launch<T, DK, 128>(a, s);
  if (units * (a.dv / 64) >= want) return launch<T, DK, 64>(a, s);
  return launch<T, DK, 32>(a, s);
}

}  // namespace

cudaError_t launch_decay_step(const DecayStep& a, lizard_dtype dt, cudaStream_t s, int* launches) {
  trace_begin("decay_step", s);
  cudaError_t e;
  if (dt == LIZARD_F32)
    e = a.dk == 64 ? dispatch<float, 64>(a, s) : dispatch<float, 128>(a, s);
  else
    e = a.dk == 64 ? dispatch<bf16, 64>(a, s) : dispatch<bf16, 128>(a, s);
  trace_end(s);
  ++*launches;
  return e;
}

}  // namespace lz
