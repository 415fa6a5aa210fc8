// k_decay_simt.cu -- one pass of the linear attention with a decay per head on CUDA cores, for fp32
// (and for what the tensor-core pass does not take), the sum over the heads of a group, and the
// gradient of log_decay from the passes' sums.
//   out_o = sum_s D(o, s) (a_o . b_s) c_s + (decay from the chunk's edge) a_o^T H,
// chunk after chunk of 64 tokens in the pass's direction, H the state that enters the chunk.  A CTA
// takes 64 of c's channels of one head; H, the chunk's rows and its scores stay in shared memory,
// every product is fp32 with 4 x 4 (or 8 x 4) results a thread.
#include "lizard_dev.cuh"
#include "lizard_internal.h"

namespace lz {
namespace {

constexpr int kC = kDecayChunk;  // tokens of a chunk
constexpr int kDc = kDecaySlice;  // channels of c of a CTA
constexpr int kThreads = 256;
constexpr int kSp = kC + 4;  // pitch of the scores

template <int DA>
struct Smem {
  static constexpr int P = DA + 4;
  float a[kC][P], b[kC][P], c[kC][kDc], s[kC][kSp], h[DA][kDc];
  float hi[kC], lo[kC];    // the sum of log_decay up to each token (its finite part) in two floats
  int doc[kC];             // documents begun up to each token
  float in[kC], out[kC];   // decays from before the chunk to each token, from each token to the end
  float diag[kC];
  float all;               // decay of the whole chunk
};

// Rows t0 .. t0 + 63 of d channels (the pitch of dst is its own) as fp32; zeros from `end` on.
template <typename T, int P>
__device__ __forceinline__ void load_rows(float (*dst)[P], const T* src, int64_t st, int t0, int end, int d) {
  const int quads = d / 4;
  for (int i = threadIdx.x; i < kC * quads; i += kThreads) {
    const int r = i / quads, q = i - r * quads;
    const float4 v = t0 + r < end ? ld4(src + (int64_t)(t0 + r) * st + 4 * q) : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(&dst[r][4 * q]) = v;
  }
}

// The chunk's decays, by one warp: two tokens a lane, sums in 64 bits so that differences of far
// sums keep their digits.
template <int DA>
__device__ __forceinline__ void decays(Smem<DA>& m, const float* lg, int64_t st, int t0, int end) {
  const int lane = threadIdx.x;
  double x[2];
  int n[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = t0 + 2 * lane + k;
    const float g = t < end ? lg[t * st] : 0.f;
    n[k] = g < kDecayNone;
    x[k] = n[k] ? 0.0 : (double)g;
  }
  double sum = x[0] + x[1];
  int docs = n[0] + n[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, sum, o);
    const int v = __shfl_up_sync(0xffffffffu, docs, o);
    if (lane >= o) sum += u, docs += v;
  }
  const double total = __shfl_sync(0xffffffffu, sum, 31);
  const int last = __shfl_sync(0xffffffffu, docs, 31);
  const double b[2] = {sum - x[1], sum};
  const int dc[2] = {docs - n[1], docs};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 2 * lane + k;
    m.hi[i] = (float)b[k];
    m.lo[i] = (float)(b[k] - (double)m.hi[i]);
    m.doc[i] = dc[k];
    m.in[i] = dc[k] ? 0.f : expf((float)b[k]);
    m.out[i] = dc[k] != last ? 0.f : expf((float)(total - b[k]));
  }
  if (lane == 0) m.all = last ? 0.f : expf((float)total);
}

template <typename T, int DA>
__global__ void __launch_bounds__(kThreads) decay_simt_kernel(DecayPass a, DecaySegs g) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem<DA>& m = *reinterpret_cast<Smem<DA>*>(raw);
  pdl_wait();
  const int tid = threadIdx.x, tc = tid % 16, ti = tid / 16;
  const int slices = a.dc / kDc, units = a.B * a.H;
  const int slice = blockIdx.x % slices, unit = blockIdx.x / slices % units, seg = blockIdx.x / slices / units;
  const int n = unit / a.H, h = unit - n * a.H, c0 = slice * kDc;
  int count = a.L;
  if (a.count) {
    count = a.count[n];
    if (count < 0 || count > a.L) {
      if (tid == 0) raise_status(a.status, kDevCheck);
      count = 0;
    }
  }
  const T* pa = static_cast<const T*>(a.a) + n * a.sa.n + h / a.ga * a.sa.h;
  const T* pb = static_cast<const T*>(a.b) + n * a.sb.n + h / a.gb * a.sb.h;
  const T* pc = static_cast<const T*>(a.c) + n * a.sc.n + h / a.gc * a.sc.h + c0;
  const T* px = a.x ? static_cast<const T*>(a.x) + n * a.sx.n + h / a.gx * a.sx.h + c0 : nullptr;
  const float* lg = a.lg + n * a.sg.n + h * a.sg.h;
  const int64_t so = n * a.so.n + h * a.so.h + c0;
  auto put = [&](int t, int col, float4 v) {
    if (a.out_f32)
      st4(static_cast<float*>(a.out) + so + t * a.so.t + col, v);
    else
      st4(static_cast<T*>(a.out) + so + t * a.so.t + col, v);
  };
  // element (i, j) of the state of this head
  auto state = [&](int i, int j) {
    return (int64_t)unit * DA * a.dc + (a.state_t ? (int64_t)(c0 + j) * DA + i : (int64_t)i * a.dc + c0 + j);
  };
  float* seg_h = g.seg_h + (((int64_t)seg * units + unit) * slices + slice) * DA * kDc;
  for (int e = tid; e < DA * kDc; e += kThreads) {
    const int i = a.state_t ? e % DA : e / kDc, j = a.state_t ? e / DA : e % kDc;
    if (g.segs > 1)
      m.h[e / kDc][e % kDc] = g.states_only ? 0.f : seg_h[e];
    else
      m.h[i][j] = a.init ? a.init[state(i, j)] : 0.f;
  }
  float* dots[2] = {nullptr, nullptr};
  if (px) {
    const int64_t o = ((int64_t)slice * a.B * a.H + unit) * a.L;
    dots[0] = a.dot_in + o, dots[1] = a.dot_out + o;
  }
  // this segment's chunks, in the pass's order
  const int chunks = (count + kC - 1) / kC, done = min(seg * g.cps, chunks), num = min(g.cps, chunks - done);
  float product = 1.f;
  for (int step = done; step < done + num; ++step) {
    const int t0 = (a.rev ? chunks - 1 - step : step) * kC;
    if (!g.states_only) load_rows<T>(m.a, pa, a.sa.t, t0, count, DA);
    load_rows<T>(m.b, pb, a.sb.t, t0, count, DA);
    load_rows<T>(m.c, pc, a.sc.t, t0, count, kDc);
    if (tid < 32) decays(m, lg, a.sg.t, t0, count);
    __syncthreads();
    const float* from_state = a.rev ? m.out : m.in;  // from the state that enters to each token
    const float* to_state = a.rev ? m.in : m.out;    // from each token to the state that leaves
    product *= m.all;
    if (!g.states_only) {
    // scores with their decays; the diagonal apart
    float acc[4][4] = {};
#pragma unroll 4
    for (int k = 0; k < DA; k += 4) {
      float4 x[4], y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = *reinterpret_cast<const float4*>(&m.a[ti + 16 * r][k]);
        y[r] = *reinterpret_cast<const float4*>(&m.b[tc + 16 * r][k]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[r][c] = fmaf(x[r].x, y[c].x, acc[r][c]);
          acc[r][c] = fmaf(x[r].y, y[c].y, acc[r][c]);
          acc[r][c] = fmaf(x[r].z, y[c].z, acc[r][c]);
          acc[r][c] = fmaf(x[r].w, y[c].w, acc[r][c]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int o = ti + 16 * r, s = tc + 16 * c;
        const int late = a.rev ? s : o, early = a.rev ? o : s;
        float d = 0.f;
        if (late > early && m.doc[late] == m.doc[early])
          d = expf((m.hi[late] - m.hi[early]) + (m.lo[late] - m.lo[early]));
        m.s[o][s] = d > 0.f ? acc[r][c] * a.scale_in * d : 0.f;
        if (o == s) m.diag[o] = acc[r][c] * a.scale_in;
      }
    __syncthreads();
    // out = scores c + decay a^T H
    float in[4][4] = {}, st[4][4] = {};
#pragma unroll 4
    for (int j = 0; j < kC; j += 4) {
      float4 x[4], y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = *reinterpret_cast<const float4*>(&m.s[ti + 16 * r][j]);
        y[r] = *reinterpret_cast<const float4*>(&m.c[j + r][4 * tc]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          in[r][0] = fmaf(w[q], y[q].x, in[r][0]);
          in[r][1] = fmaf(w[q], y[q].y, in[r][1]);
          in[r][2] = fmaf(w[q], y[q].z, in[r][2]);
          in[r][3] = fmaf(w[q], y[q].w, in[r][3]);
        }
      }
    }
#pragma unroll 4
    for (int j = 0; j < DA; j += 4) {
      float4 x[4], y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = *reinterpret_cast<const float4*>(&m.a[ti + 16 * r][j]);
        y[r] = *reinterpret_cast<const float4*>(&m.h[j + r][4 * tc]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          st[r][0] = fmaf(w[q], y[q].x, st[r][0]);
          st[r][1] = fmaf(w[q], y[q].y, st[r][1]);
          st[r][2] = fmaf(w[q], y[q].z, st[r][2]);
          st[r][3] = fmaf(w[q], y[q].w, st[r][3]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int o = ti + 16 * r, t = t0 + o;
      const float e = from_state[o];
#pragma unroll
      for (int q = 0; q < 4; ++q) st[r][q] = e > 0.f ? e * st[r][q] : 0.f;
      if (px) {
        const float4 x = t < count ? ld4(px + t * a.sx.t + 4 * tc) : make_float4(0.f, 0.f, 0.f, 0.f);
        float d0 = x.x * in[r][0] + x.y * in[r][1] + x.z * in[r][2] + x.w * in[r][3];
        float d1 = x.x * st[r][0] + x.y * st[r][1] + x.z * st[r][2] + x.w * st[r][3];
#pragma unroll
        for (int x16 = 8; x16 > 0; x16 >>= 1) {
          d0 += __shfl_xor_sync(0xffffffffu, d0, x16);
          d1 += __shfl_xor_sync(0xffffffffu, d1, x16);
        }
        if (tc == 0 && t < count) dots[0][t] = a.scale_out * d0, dots[1][t] = a.scale_out * d1;
      }
      const float4 cd = *reinterpret_cast<const float4*>(&m.c[o][4 * tc]);
      const float dg = m.diag[o];
      if (t < count)
        put(t, 4 * tc, make_float4(a.scale_out * (fmaf(dg, cd.x, in[r][0]) + st[r][0]),
                                   a.scale_out * (fmaf(dg, cd.y, in[r][1]) + st[r][1]),
                                   a.scale_out * (fmaf(dg, cd.z, in[r][2]) + st[r][2]),
                                   a.scale_out * (fmaf(dg, cd.w, in[r][3]) + st[r][3])));
    }
    __syncthreads();
    }
    // H <- decay H + sum_s decay_s b_s c_s^T: rows ti * NR + r, columns 4 tc ..
    constexpr int NR = DA / 16;
    float u[NR][4];
    const float all = m.all;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float4 x = *reinterpret_cast<const float4*>(&m.h[ti * NR + r][4 * tc]);
      u[r][0] = all > 0.f ? all * x.x : 0.f, u[r][1] = all > 0.f ? all * x.y : 0.f;
      u[r][2] = all > 0.f ? all * x.z : 0.f, u[r][3] = all > 0.f ? all * x.w : 0.f;
    }
#pragma unroll 2
    for (int s = 0; s < kC; ++s) {
      const float e = to_state[s] * a.scale_in;
      float4 y = *reinterpret_cast<const float4*>(&m.c[s][4 * tc]);
      y = e != 0.f ? make_float4(y.x * e, y.y * e, y.z * e, y.w * e) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < NR; r += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&m.b[s][ti * NR + r]);
        const float w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u[r + q][0] = fmaf(w[q], y.x, u[r + q][0]);
          u[r + q][1] = fmaf(w[q], y.y, u[r + q][1]);
          u[r + q][2] = fmaf(w[q], y.z, u[r + q][2]);
          u[r + q][3] = fmaf(w[q], y.w, u[r + q][3]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
      *reinterpret_cast<float4*>(&m.h[ti * NR + r][4 * tc]) = make_float4(u[r][0], u[r][1], u[r][2], u[r][3]);
    __syncthreads();
  }
  if (g.states_only) {
    __syncthreads();  // without a chunk, zeros
    for (int e = tid; e < DA * kDc; e += kThreads) seg_h[e] = m.h[e / kDc][e % kDc];
    if (tid == 0) g.seg_d[((int64_t)seg * units + unit) * slices + slice] = product;
    return;
  }
  // rows behind the sequence, each segment its share of the axis
  const int z0 = max(count, (int)min((int64_t)seg * g.cps * kC, (int64_t)a.L)),
            z1 = (int)min((int64_t)(seg + 1) * g.cps * kC, (int64_t)a.L);
  for (int64_t i = tid; i < (int64_t)(z1 - z0) * (kDc / 4); i += kThreads)
    put(z0 + (int)(i / (kDc / 4)), 4 * (int)(i % (kDc / 4)), make_float4(0.f, 0.f, 0.f, 0.f));
  if (a.fin && seg == g.segs - 1) {
    __syncthreads();  // without a chunk, the initial state
    for (int e = tid; e < DA * kDc; e += kThreads) {
      const int i = a.state_t ? e % DA : e / kDc, j = a.state_t ? e / DA : e % kDc;
      a.fin[state(i, j)] = m.h[i][j];
    }
  }
}

// The segments' starting states in place of their own states: cur = init; for each segment its slot
// becomes cur, and cur = decay cur + the segment's state.  A thread has one element of a head's state;
// eight segments' states are on their way at a time.
__global__ void __launch_bounds__(256) decay_join_kernel(DecayPass p, DecaySegs g) {
  pdl_wait();
  const int slices = p.dc / kDc, per = p.da * kDc;
  const int us = blockIdx.x / (per / 256), e = (blockIdx.x - us * (per / 256)) * 256 + threadIdx.x;
  const int unit = us / slices, i = e / kDc, c = (us - unit * slices) * kDc + e % kDc;
  const int64_t total = (int64_t)p.B * p.H * slices, at = (int64_t)us * per + e;
  float cur = p.init ? p.init[(int64_t)unit * p.da * p.dc + (p.state_t ? c * p.da + i : i * p.dc + c)] : 0.f;
  for (int s0 = 0; s0 < g.segs; s0 += 8) {
    float own[8], d[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool has = s0 + k + 1 < g.segs;
      own[k] = has ? g.seg_h[(s0 + k) * total * per + at] : 0.f;
      d[k] = has ? g.seg_d[(s0 + k) * total + us] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (s0 + k < g.segs) g.seg_h[(s0 + k) * total * per + at] = cur;
      cur = fmaf(d[k], cur, own[k]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) decay_heads_kernel(int Hk, int G, int L, int d, const float* part, T* out,
                                                               Strides so, int64_t quads) {
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= quads) return;
  const int per = d / 4;
  const int64_t row = i / per;
  const int c = 4 * (int)(i - row * per);
  const int64_t u = row / L;
  const int t = (int)(row - u * L), n = (int)(u / Hk), h = (int)(u - (int64_t)n * Hk);
  const float* p = part + (u * G * L + t) * d + c;
  float4 s = ld4(p);
  for (int g = 1; g < G; ++g) {
    const float4 x = ld4(p + (int64_t)g * L * d);
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
  }
  st4(out + n * so.n + h * so.h + t * so.t + c, s);
}

// d log_decay_t = g_t <h_{t-1}, dh_t>: the sum of all products that pass over token t.  With, for
// each token, what it receives from (rows) and gives to (cols) other tokens of its chunk and the
// states at the chunk's ends,
//   = sum_{i >= t} row_in_i - sum_{j >= t} col_in_j        within the chunk (t's own pair cancels)
//   + sum_{i >= t} row_out_i + sum_{j < t} col_out_j       between the chunk and what lies around it
//   + through                                              from before the chunk to after it.
// `through` of the chunks follows from the pairs over the edge before the first one, <h0, d_h0>:
//   edge after = through + sum col_out,  through = edge before - sum row_out  (0 where a document
// starts in the chunk).  Sums over chunks run in 64 bits, within 32 tokens in trees of fp32 (64-bit
// additions are what this GPU has least of: with them throughout, 49 us against 13 for 64 heads x 4096
// tokens).  First a warp for each chunk takes its sums of row_out
// and col_out and whether a document starts, and a block for each head <h0, d_h0>; then a warp for
// each chunk adds up the edge in front of it and writes its tokens.
__device__ __forceinline__ double warp_sum64(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ int gate_count(const DecayGate& a, int n) {
  const int c = a.count ? a.count[n] : a.L;
  return c < 0 || c > a.L ? 0 : c;
}

constexpr int kGateWarps = 4;
// sums [units][chunks + 1]: of the chunks (x: rows, y: cols; a start as rows = NaN), then <h0, d_h0>
__global__ void __launch_bounds__(32 * kGateWarps) decay_gate_sums_kernel(DecayGate a, int chunks) {
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int units = a.B * a.H, per = (chunks + kGateWarps - 1) / kGateWarps;
  if (blockIdx.x < units) {
    double s = 0.0;
    if (a.h0) {
      const float4* x = reinterpret_cast<const float4*>(a.h0 + (int64_t)blockIdx.x * a.state);
      const float4* y = reinterpret_cast<const float4*>(a.d_h0 + (int64_t)blockIdx.x * a.state);
#pragma unroll 4
      for (int i = threadIdx.x; i < a.state / 4; i += 32 * kGateWarps) {
        const float4 u = x[i], v = y[i];
        s += (double)(u.x * v.x) + (double)(u.y * v.y) + (double)(u.z * v.z) + (double)(u.w * v.w);
      }
    }
    __shared__ double part[kGateWarps];
    s = warp_sum64(s);
    if (lane == 0) part[warp] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < kGateWarps; ++w) s += part[w];
    if (threadIdx.x == 0) a.sums[(int64_t)blockIdx.x * (chunks + 1) + chunks] = make_double2(s, 0.0);
    return;
  }
  const int unit = (blockIdx.x - units) / per, c = (blockIdx.x - units - unit * per) * kGateWarps + warp;
  const int n = unit / a.H, h = unit - n * a.H;
  const int t0 = c * a.chunk, end = min(t0 + a.chunk, gate_count(a, n));
  if (t0 >= end) return;
  const int64_t plane = (int64_t)units * a.L, base = (int64_t)unit * a.L;
  const float* lg = a.lg + n * a.sg.n + h * a.sg.h;
  float r = 0.f, c1 = 0.f;
  bool start = false;
#pragma unroll 4
  for (int t = t0 + lane; t < end; t += 32) {
#pragma unroll 4
    for (int s = 0; s < a.out_slices; ++s) r += a.row_out[s * plane + base + t], c1 += a.col_out[s * plane + base + t];
    start |= lg[t * a.sg.t] < kDecayNone;
  }
  const double rows = warp_sum(r), cols = warp_sum(c1);
  start = __any_sync(0xffffffffu, start);
  if (lane == 0) a.sums[(int64_t)unit * (chunks + 1) + c] = make_double2(start ? nan("") : rows, cols);
}

__global__ void __launch_bounds__(32 * kGateWarps) decay_gate_kernel(DecayGate a, int chunks) {
  pdl_wait();
  const int lane = threadIdx.x % 32, per = (chunks + kGateWarps - 1) / kGateWarps;
  const int unit = blockIdx.x / per, c = (blockIdx.x - unit * per) * kGateWarps + threadIdx.x / 32;
  if (c >= chunks) return;
  const int n = unit / a.H, h = unit - n * a.H, count = gate_count(a, n);
  const int t0 = c * a.chunk, end = min(t0 + a.chunk, count);
  const int64_t plane = (int64_t)a.B * a.H * a.L, base = (int64_t)unit * a.L;
  for (int t = max(t0, count) + lane; t < min(t0 + a.chunk, a.L); t += 32) a.d_lg[base + t] = 0.f;
  if (t0 >= end) return;
  // the edge in front of the chunk: 32 chunks at a time, from the last start on
  const double2* sums = a.sums + (int64_t)unit * (chunks + 1);
  double edge = sums[chunks].x;
  for (int k = 0; k < c; k += 32) {
    double2 s = make_double2(0.0, 0.0);
    if (k + lane < c) s = sums[k + lane];
    const unsigned starts = __ballot_sync(0xffffffffu, isnan(s.x));
    const int last = 31 - __clz(starts);  // -1: none
    if (starts) edge = 0.0;
    edge += warp_sum64(lane < last ? 0.0 : lane == last ? s.y : s.y - s.x);
  }
  const double2 own = sums[c];
  const double through = isnan(own.x) ? 0.0 : edge - own.x;
  const float* lg = a.lg + n * a.sg.n + h * a.sg.h;
  // the chunk's groups of 32 tokens: all of their numbers first, then from the last group to the first
  // with what lies behind each
  constexpr int kG = kDecayTile / 32;
  static_assert(kDecayTile >= kDecayChunk && kDecayTile % 32 == 0, "groups of a chunk");
  float sum[kG], col[kG];
  unsigned cut = 0;  // a document's start: nothing passes over it
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    const int t = t0 + 32 * g + lane;
    sum[g] = col[g] = 0.f;
    if (t < end) {
      if (lg[t * a.sg.t] < kDecayNone) cut |= 1u << g;
#pragma unroll 2
      for (int s = 0; s < a.in_slices; ++s)
        sum[g] += a.row_in[s * plane + base + t] - (a.col_in ? a.col_in[s * plane + base + t] : 0.f);
#pragma unroll 4
      for (int s = 0; s < a.out_slices; ++s)
        sum[g] += a.row_out[s * plane + base + t], col[g] += a.col_out[s * plane + base + t];
    }
  }
  double behind = through, before = own.y;  // the suffix sums behind a group; col_out of the tokens before its end
#pragma unroll
  for (int g = kG - 1; g >= 0; --g) {
    const int t = t0 + 32 * g + lane;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float u = __shfl_down_sync(0xffffffffu, sum[g], o), v = __shfl_down_sync(0xffffffffu, col[g], o);
      if (lane + o < 32) sum[g] += u, col[g] += v;
    }
    if (t < end) a.d_lg[base + t] = cut >> g & 1 ? 0.f : (float)(behind + before + (double)(sum[g] - col[g]));
    behind += __shfl_sync(0xffffffffu, sum[g], 0);
    before -= __shfl_sync(0xffffffffu, col[g], 0);
  }
}

template <typename T, int DA>
cudaError_t launch(const DecayPass& a, const DecaySegs& g, int64_t blocks, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(decay_simt_kernel<T, DA>, sizeof(Smem<DA>), done);
  if (e != cudaSuccess) return e;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_pdl(decay_simt_kernel<T, DA>, dim3((unsigned)blocks), dim3(kThreads), sizeof(Smem<DA>), s, a, g);
}

cudaError_t dispatch(const DecayPass& a, lizard_dtype dt, const DecaySegs& g, int64_t blocks, cudaStream_t s) {
  if (dt == LIZARD_F32)
    return a.da == 64 ? launch<float, 64>(a, g, blocks, s) : launch<float, 128>(a, g, blocks, s);
  return a.da == 64 ? launch<bf16, 64>(a, g, blocks, s) : launch<bf16, 128>(a, g, blocks, s);
}

// One CTA an SM at da = 128, two at 64, by their shared memory; a state pass is a third of the work.
int simt_segments(int64_t ctas, int L, int da) {
  return decay_segments(ctas, da == 64 ? 304 : 152, (L + kC - 1) / kC, 0.35, 0.4);
}

}  // namespace

int decay_segments(int64_t ctas, int per_wave, int chunks, double part, double extra) {
  if (ctas >= 8 * per_wave) return 1;
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= 64 && s <= chunks; ++s) {
    const int cps = (chunks + s - 1) / s;
    if (s > 1 && (chunks + cps - 1) / cps < s) continue;  // some would be empty
    double t = (double)((ctas * s + per_wave - 1) / per_wave) * cps;
    if (s > 1) t += part * (double)((ctas * (s - 1) + per_wave - 1) / per_wave) * cps + extra;
    if (t < least) least = t, best = s;
  }
  return best;
}

size_t decay_seg_bytes(int segs, int64_t ctas, int da) {
  return segs > 1 ? (size_t)segs * ctas * ((size_t)da * kDc + 1) * sizeof(float) : 0;
}

cudaError_t launch_decay_join(const DecayPass& a, const DecaySegs& g, cudaStream_t s, int* launches) {
  const int64_t blocks = (int64_t)a.B * a.H * (a.dc / kDc) * (a.da * kDc / 256);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  trace_begin("decay_join", s);
  const cudaError_t e = launch_pdl(decay_join_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, g);
  trace_end(s);
  ++*launches;
  return e;
}

size_t decay_simt_workspace(int B, int H, int L, int da, int dc) {
  const int64_t ctas = (int64_t)B * H * (dc / kDc);
  return decay_seg_bytes(simt_segments(ctas, L, da), ctas, da);
}

cudaError_t launch_decay_simt(const DecayPass& a, lizard_dtype dt, float* ws, cudaStream_t s, int* launches) {
  const int64_t ctas = (int64_t)a.B * a.H * (a.dc / kDc);
  const int chunks = (a.L + kC - 1) / kC;
  DecaySegs g{};
  g.segs = simt_segments(ctas, a.L, a.da);
  g.cps = chunks ? (chunks + g.segs - 1) / g.segs : 1;
  if (g.segs > 1) {
    g.seg_h = ws, g.seg_d = ws + (size_t)g.segs * ctas * a.da * kDc;
    DecaySegs f = g;
    f.states_only = true;
    trace_begin("decay_states", s);
    cudaError_t e = dispatch(a, dt, f, ctas * (g.segs - 1), s);
    trace_end(s);
    ++*launches;
    if (e == cudaSuccess) e = launch_decay_join(a, g, s, launches);
    if (e != cudaSuccess) return e;
  }
  trace_begin("decay_simt", s);
  const cudaError_t e = dispatch(a, dt, g, ctas * g.segs, s);
  trace_end(s);
  ++*launches;
  return e;
}

cudaError_t launch_decay_heads(int B, int Hk, int G, int L, int d, const float* part, void* out, Strides so,
                               lizard_dtype dt, cudaStream_t s, int* launches) {
  const int64_t quads = (int64_t)B * Hk * L * (d / 4), blocks = (quads + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  trace_begin("decay_heads", s);
  const cudaError_t e =
      dt == LIZARD_F32
          ? launch_pdl(decay_heads_kernel<float>, dim3((unsigned)blocks), dim3(kThreads), 0, s, Hk, G, L, d, part,
                       static_cast<float*>(out), so, quads)
          : launch_pdl(decay_heads_kernel<bf16>, dim3((unsigned)blocks), dim3(kThreads), 0, s, Hk, G, L, d, part,
                       static_cast<bf16*>(out), so, quads);
  trace_end(s);
  ++*launches;
  return e;
}

cudaError_t launch_decay_gate(const DecayGate& a, cudaStream_t s, int* launches) {
  const int chunks = (a.L + a.chunk - 1) / a.chunk;
  const int64_t units = (int64_t)a.B * a.H, blocks = units * ((chunks + kGateWarps - 1) / kGateWarps);
  if (units + blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  trace_begin("decay_gate_sums", s);
  cudaError_t e = launch_pdl(decay_gate_sums_kernel, dim3((unsigned)(units + blocks)), dim3(32 * kGateWarps), 0, s, a, chunks);
  trace_end(s);
  ++*launches;
  if (e != cudaSuccess) return e;
  trace_begin("decay_gate", s);
  e = launch_pdl(decay_gate_kernel, dim3((unsigned)blocks), dim3(32 * kGateWarps), 0, s, a, chunks);
  trace_end(s);
  ++*launches;
  return e;
}

size_t decay_gate_workspace(int B, int H, int L, int chunk) {
  return (size_t)B * H * ((L + chunk - 1) / chunk + 1) * sizeof(double2);
}

}  // namespace lz
