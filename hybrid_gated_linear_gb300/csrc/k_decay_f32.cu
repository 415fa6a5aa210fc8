// k_decay_f32.cu -- one pass of the linear attention with a decay per head in fp32 (and for the bf16 rows that
// the tensor-memory pass does not take), the join of segments, the sum over the heads of a group, and the
// gradient of log_decay from the passes' sums.
//   out_o = sum_s D(o, s) (a_o . b_s) c_s + (decay from the chunk's edge) a_o^T H,
// chunk after chunk of 64 tokens in the pass's direction, H the state that enters the chunk.  A CTA takes
// 64 of c's channels of one head; the chunk's rows, its scores and H lie in shared memory in fp32.
// Every product is made of three tf32 products of the warp-level tensor instructions, x = hi + lo with hi the
// upper 11 bits: hi hi + hi lo + lo hi, which leaves 2^-22 of a product (8 more bits in each operand than
// tcgen05's bf16 parts, whose three tiles an operand would not fit beside each other).  Against 4 x 4 results a
// thread by fp32 multiply-adds: 5 sequences of 1999 tokens, 12 heads of 64 x 128, 248 -> 142 us.  Bound by the
// chain of a chunk (rows in, scores, out, state; two CTAs an SM): tensor cycles 31%, DRAM 5%.
#include "lizard_dev.cuh"
#include "lizard_internal.h"
#include "tc_sm100.cuh"

namespace lz {
namespace {

constexpr int kC = kDecayChunk;  // tokens of a chunk
constexpr int kDc = kDecaySlice;  // channels of c of a CTA
constexpr int kThreads = 256;
// Pitches: 4 more than a multiple of 32 words where a fragment's eight rows lie along the pitch, 8 more where
// its four do.
constexpr int kSp = kC + 4, kCp = kDc + 8;

template <int DA>
struct Smem {
  static constexpr int P = DA + 4;
  float a[kC][P], b[kC][P], c[kC][kCp], s[kC][kSp], h[DA][kCp];
  float hi[kC], lo[kC];    // log2 of the decays up to each token (their finite part) in two floats
  int doc[kC];             // documents begun up to each token
  float in[kC], out[kC];   // decays from before the chunk to each token, from each token to the end
  float diag[kC];          // the scores of the tokens themselves
  float dots[2][kC];       // of a row with the state: [half of the channels]
  float cols[4][kC], rows[kC];  // the products that pass over a token: see pass_over
  float all;               // decay of the whole chunk
};

// Rows t0 .. t0 + 63 of d channels (the pitch of dst is its own) as fp32; zeros from `end` on.  fp32 rows by
// asynchronous copies, all of a chunk's on their way together (rows_wait).
template <typename T, int P>
__device__ __forceinline__ void load_rows(float (*dst)[P], const T* src, int64_t st, int t0, int end, int d) {
  const int quads = d / 4;
#pragma unroll 4
  for (int i = threadIdx.x; i < kC * quads; i += kThreads) {
    const int r = i / quads, q = i - r * quads;
    if (sizeof(T) == 4) {
      const bool there = t0 + r < end;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(&dst[r][4 * q])),
                   "l"(src + (there ? (int64_t)(t0 + r) * st + 4 * q : 0)), "r"(there ? 16 : 0)
                   : "memory");
      continue;
    }
    const float4 v = t0 + r < end ? ld4(src + (int64_t)(t0 + r) * st + 4 * q) : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(&dst[r][4 * q]) = v;
  }
}

__device__ __forceinline__ void rows_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
    x[k] = n[k] ? 0.0 : (double)g * 1.4426950408889634;
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
    m.in[i] = dc[k] ? 0.f : exp2f((float)b[k]);
    m.out[i] = dc[k] != last ? 0.f : exp2f((float)(total - b[k]));
  }
  if (lane == 0) m.all = last ? 0.f : exp2f((float)total);
}

// A word as two tf32 operands, both rounded to nearest: 11 bits, and 11 of what is left.  (The instruction
// does not read a word's lower 13 bits; cut off instead of rounded, results were 1.4e-6 off, this way 7e-7, and
// with the small products' sums apart 3.5e-7.)
struct Two {
  uint32_t hi, lo;
};
__device__ __forceinline__ Two two(float x) {
  const uint32_t hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  return {hi, __float_as_uint(x - __uint_as_float(hi)) + 0x1000u};
}
// d (16 x 8) += a (16 x 8) b (8 x 8)
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// One k-step of 8 of a warp's 16 x (8 NT) results: a(row, k) and b(col, k, k / 4) give the operands' elements
// at the lane's places.  The instruction cuts its sums off at 24 bits: the small products have sums of their
// own, so that the large ones are cut once a step and not three times.
template <int NT, typename A, typename B>
__device__ __forceinline__ void step8(float (&d)[NT][4], float (&small)[NT][4], A a, B b) {
  const int g = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
  uint32_t ah[4], al[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const Two t = two(a(g + 8 * (e & 1), c + 4 * (e >> 1)));
    ah[e] = t.hi, al[e] = t.lo;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const Two b0 = two(b(8 * n + g, c, 0)), b1 = two(b(8 * n + g, c + 4, 1));
    mma_tf32(small[n], al, b0.hi, b1.hi);
    mma_tf32(small[n], ah, b0.lo, b1.lo);
    mma_tf32(d[n], ah, b0.hi, b1.hi);
  }
}
template <int NT>
__device__ __forceinline__ void join_small(float (&d)[NT][4], float (&small)[NT][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[n][e] += small[n][e], small[n][e] = 0.f;
}

// The products W_is of a chunk's rows i and columns s < i that pass over each token t, s < t <= i, summed from
// W in the scores' layout: E_it = sum_{s < t} W_is by running sums along the 32 columns of a warp, of which the
// rows from t on are added up into cols[rows / 16][t]; rows[i] keeps the sum over the first 32 columns, which
// all of the others have before them.  No product on one side of t enters, not even to be taken off again.
template <int DA>
__device__ __forceinline__ void pass_over(Smem<DA>& m, float (&w)[4][4], int r0, int n0) {
  const int lane = threadIdx.x & 31, gr = lane >> 2, cq = 2 * (lane & 3);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int o = r0 + gr + 8 * q;
    float run = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float w0 = w[e][2 * q], pair = w0 + w[e][2 * q + 1];
      float to = pair;  // with the lanes before
#pragma unroll
      for (int k = 1; k < 4; k <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, to, k, 4);
        if ((lane & 3) >= k) to += u;
      }
      float before = __shfl_up_sync(0xffffffffu, to, 1, 4);
      if ((lane & 3) == 0) before = 0.f;
      before += run;
      const int t = n0 + 8 * e + cq;
      w[e][2 * q] = o >= t ? before : 0.f;
      w[e][2 * q + 1] = o > t ? before + w0 : 0.f;
      run += __shfl_sync(0xffffffffu, to, 3, 4);
    }
    if (n0 == 0 && (lane & 3) == 0) m.rows[o] = run;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float c = w[e][b] + w[e][2 + b];
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) c += __shfl_xor_sync(0xffffffffu, c, k);
      if (gr == 0) m.cols[r0 >> 4][n0 + 8 * e + cq + b] = c;
    }
}
// Two warps, behind a barrier: the sum of token t.
template <int DA>
__device__ __forceinline__ float passed(const Smem<DA>& m, int t) {
  float d = 0.f;
  if (t >= 32) {  // the first 32 columns of the rows from t on
    d = m.rows[t];
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const float u = __shfl_down_sync(0xffffffffu, d, k);
      if ((t & 31) + k < 32) d += u;
    }
  }
  for (int r = t >> 4; r < 4; ++r) d += m.cols[r][t];
  return d;
}

// Warp w of eight: rows 16 (w mod 4) .. of the chunk's 64, columns 32 (w / 4) .. of 64; of the state the rows
// DA / 4 (w mod 4) ...  A lane's results of tile n: rows g, g + 8, columns 8 n + 2 c, + 1.
// GATE: the passes that the gradient of log_decay is made from (a.x is there).
template <typename T, int DA, bool GATE>
__global__ void __launch_bounds__(kThreads) decay_f32_kernel(DecayPass a, DecaySegs g) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem<DA>& m = *reinterpret_cast<Smem<DA>*>(raw);
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const T* px = GATE ? static_cast<const T*>(a.x) + n * a.sx.n + h / a.gx * a.sx.h + c0 : nullptr;
  const int edges = (a.L + kC - 1) / kC;  // chunks of the axis, each with a state that enters it
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
  const int64_t dot0 = ((int64_t)slice * units + unit) * a.L;
  const int r0 = 16 * (warp & 3), n0 = 32 * (warp >> 2), gr = lane >> 2, cq = 2 * (lane & 3);
  constexpr int MT = DA / 64;  // 16-row tiles of the state of a warp
  const int h0 = 16 * MT * (warp & 3);
  // this segment's chunks, in the pass's order
  const int chunks = (count + kC - 1) / kC, done = min(seg * g.cps, chunks), num = min(g.cps, chunks - done);
  float product = 1.f;
  for (int step = done; step < done + num; ++step) {
    const int t0 = (a.rev ? chunks - 1 - step : step) * kC;
    if (!g.states_only) load_rows<T>(m.a, pa, a.sa.t, t0, count, DA);
    load_rows<T>(m.b, pb, a.sb.t, t0, count, DA);
    load_rows<T>(m.c, pc, a.sc.t, t0, count, kDc);
    if (tid < 32) decays(m, lg, a.sg.t, t0, count);
    rows_wait();
    __syncthreads();
    const float* from_state = a.rev ? m.out : m.in;  // from the state that enters to each token
    const float* to_state = a.rev ? m.in : m.out;    // from each token to the state that leaves
    product *= m.all;
    if (!g.states_only) {
      // scores with their decays: the chunk's half on the pass's side of the diagonal, and that apart (the
      // token's own pair passes over no decay)
      if (a.rev ? n0 + 31 >= r0 : n0 <= r0 + 15) {
        float acc[4][4] = {}, small[4][4] = {};
#pragma unroll 2
        for (int k = 0; k < DA; k += 8)
          step8(acc, small, [&](int r, int c) { return m.a[r0 + r][k + c]; }, [&](int r, int c, int) { return m.b[n0 + r][k + c]; });
        join_small(acc, small);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int o = r0 + gr + 8 * (q >> 1), s = n0 + 8 * e + cq + (q & 1);
            const int late = a.rev ? s : o, early = a.rev ? o : s;
            float d = 0.f;
            if (late > early && m.doc[late] == m.doc[early])
              d = tc::ex2_approx((m.hi[late] - m.hi[early]) + (m.lo[late] - m.lo[early]));
            m.s[o][s] = d > 0.f ? acc[e][q] * a.scale_in * d : 0.f;
            if (o == s) m.diag[o] = acc[e][q] * a.scale_in;
            acc[e][q] = d > 0.f ? acc[e][q] * a.scale_in * d : 0.f;
          }
        if (GATE && a.dot_in) {
          // times this CTA's channels of x_o . c_s
          float xc[4][4] = {};
#pragma unroll 2
          for (int k = 0; k < kDc; k += 8)
            step8(xc, small,
                  [&](int r, int c) { return t0 + r0 + r < count ? ld_f(px + (int64_t)(t0 + r0 + r) * a.sx.t + k + c) : 0.f; },
                  [&](int r, int c, int) { return m.c[n0 + r][k + c]; });
          join_small(xc, small);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[e][q] *= xc[e][q];
          pass_over(m, acc, r0, n0);
        }
      }
      __syncthreads();
      // out = scores c + decay a^T H
      float in[4][4] = {}, st[4][4] = {};
      {
        float small[4][4] = {};
        const int ka = a.rev ? r0 : 0, kb = a.rev ? kC : r0 + 16;  // the other scores of these rows are 0
#pragma unroll 2
        for (int k = ka; k < kb; k += 8)
          step8(in, small, [&](int r, int c) { return m.s[r0 + r][k + c]; }, [&](int r, int c, int) { return m.c[k + c][n0 + r]; });
        join_small(in, small);
#pragma unroll 2
        for (int k = 0; k < DA; k += 8)
          step8(st, small, [&](int r, int c) { return m.a[r0 + r][k + c]; }, [&](int r, int c, int) { return m.h[k + c][n0 + r]; });
        join_small(st, small);
      }
      float dot[2] = {};  // of a row, with the state
      float2 y[4][2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int o = r0 + gr + 8 * q, t = t0 + o;
        const float e = from_state[o], dg = m.diag[o];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 u = make_float2(in[k][2 * q], in[k][2 * q + 1]);
          float2 w = make_float2(e * st[k][2 * q], e * st[k][2 * q + 1]);
          if (!(e > 0.f)) w = make_float2(0.f, 0.f);
          const int col = n0 + 8 * k + cq;
          const float2 cd = *reinterpret_cast<const float2*>(&m.c[o][col]);
          y[k][q] = make_float2(a.scale_out * (fmaf(dg, cd.x, u.x) + w.x), a.scale_out * (fmaf(dg, cd.y, u.y) + w.y));
          if (GATE && t < count) {
            float x0, x1;
            if (sizeof(T) == 4) {
              const float2 v = *reinterpret_cast<const float2*>(px + t * a.sx.t + col);
              x0 = v.x, x1 = v.y;
            } else {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(px + t * a.sx.t + col);
              x0 = __uint_as_float(v << 16), x1 = __uint_as_float(v & 0xffff0000u);
            }
            dot[q] += x0 * w.x + x1 * w.y;
          }
        }
      }
      if (GATE) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          dot[q] += __shfl_xor_sync(0xffffffffu, dot[q], 1);
          dot[q] += __shfl_xor_sync(0xffffffffu, dot[q], 2);
          if ((lane & 3) == 0) m.dots[warp >> 2][r0 + gr + 8 * q] = dot[q];
        }
      }
      __syncthreads();  // the scores and H have been read
      if (GATE && tid < kC) {
        if (t0 + tid < count) a.dot_out[dot0 + t0 + tid] = a.scale_out * (m.dots[0][tid] + m.dots[1][tid]);
      } else if (GATE && tid < 2 * kC && a.dot_in) {
        const int o = tid - kC;
        const float d = passed(m, o);
        if (t0 + o < count) a.dot_in[dot0 + t0 + o] = a.scale_out * d;
      }
      // the rows of out through the scores' place
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<float2*>(&m.s[r0 + gr + 8 * q][n0 + 8 * k + cq]) = y[k][q];
    }
    // H <- decay H + sum_s decay_s b_s c_s^T
    const float all = m.all;
    float over = 0.f;  // <H, the state that enters from the other side>, where that was kept
    float2* edge = GATE ? reinterpret_cast<float2*>(a.edge) +
                              (((int64_t)unit * edges + t0 / kC) * slices + slice) * (DA * kDc / 2) + tid
                        : nullptr;
#pragma unroll 1
    for (int r = 0; r < MT; ++r) {
      float u[4][4] = {}, small[4][4] = {};
#pragma unroll 2
      for (int k = 0; k < kC; k += 8) {
        float w[2];  // of the lane's two tokens
#pragma unroll
        for (int e = 0; e < 2; ++e) w[e] = to_state[k + (lane & 3) + 4 * e] * a.scale_in;
        step8(u, small, [&](int i, int c) { return m.b[k + c][h0 + 16 * r + i]; },
              [&](int j, int c, int e) { return w[e] * m.c[k + c][n0 + j]; });
      }
      join_small(u, small);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float2* at = reinterpret_cast<float2*>(&m.h[h0 + 16 * r + gr + 8 * q][n0 + 8 * k + cq]);
          if (GATE) {
            float2* kept = edge + ((r * 4 + k) * 2 + q) * kThreads;
            if (a.through) {
              const float2 v = *kept;
              over = fmaf(at->x, v.x, fmaf(at->y, v.y, over));
            } else {
              *kept = *at;
            }
          }
          const float2 x = all > 0.f ? *at : make_float2(0.f, 0.f);
          *at = make_float2(fmaf(all, x.x, u[k][2 * q]), fmaf(all, x.y, u[k][2 * q + 1]));
        }
    }
    if (GATE && a.through) {
      over = warp_sum(over);
      if (lane == 0)
        a.through[(((int64_t)unit * edges + t0 / kC) * slices + slice) * kDecayEdgeWarps + warp] = all > 0.f ? all * over : 0.f;
    }
    __syncthreads();
    if (!g.states_only) {
      for (int i = tid; i < kC * (kDc / 4); i += kThreads) {
        const int o = i / (kDc / 4), c = 4 * (i % (kDc / 4));
        if (t0 + o < count) put(t0 + o, c, *reinterpret_cast<const float4*>(&m.s[o][c]));
      }
      // (the next chunk's scores are written behind its first barrier)
    }
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

// d log_decay_t = g_t <h_{t-1}, dh_t>: the sum of all products that pass over token t,
//   inside_t                         between two tokens of its chunk
//   + sum_{i >= t} row_out_i         from the state before the chunk to its tokens
//   + sum_{j < t} col_out_j          from its tokens to the state behind it
//   + through                        from before the chunk to behind it.
// Each sum holds what passes over t and nothing else, and `through` comes from the states themselves, so the
// rounding of products that do not reach t stays out, however large they are (a running sum of all rows less
// all columns would carry it on behind them, where they have decayed to nothing).  A start of a document makes
// every product over it exactly 0.  A warp for each chunk: its sums over 32 tokens in trees of fp32.
__device__ __forceinline__ int gate_count(const DecayGate& a, int n) {
  const int c = a.count ? a.count[n] : a.L;
  return c < 0 || c > a.L ? 0 : c;
}

constexpr int kGateWarps = 4;
// IN, OUT: planes; all of a chunk's numbers are on their way together.
template <int IN, int OUT>
__global__ void __launch_bounds__(32 * kGateWarps) decay_gate_kernel(DecayGate a, int chunks) {
  pdl_wait();
  const int lane = threadIdx.x % 32, per = (chunks + kGateWarps - 1) / kGateWarps;
  const int unit = blockIdx.x / per, c = (blockIdx.x - unit * per) * kGateWarps + threadIdx.x / 32;
  if (c >= chunks) return;
  const int n = unit / a.H, count = gate_count(a, n);
  const int t0 = c * a.chunk, end = min(t0 + a.chunk, count);
  const int64_t plane = (int64_t)a.B * a.H * a.L, base = (int64_t)unit * a.L;
  for (int t = max(t0, count) + lane; t < min(t0 + a.chunk, a.L); t += 32) a.d_lg[base + t] = 0.f;
  if (t0 >= end) return;
  constexpr int kG = kDecayTile / 32;
  static_assert(kDecayTile >= kDecayChunk && kDecayTile % 32 == 0, "groups of a chunk");
  float in[kG], row[kG], col[kG];
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    const int t = t0 + 32 * g + lane;
    in[g] = row[g] = col[g] = 0.f;
    if (t < end) {
#pragma unroll
      for (int s = 0; s < IN; ++s) in[g] += a.inside[s * plane + base + t];
#pragma unroll
      for (int s = 0; s < OUT; ++s) row[g] += a.row_out[s * plane + base + t], col[g] += a.col_out[s * plane + base + t];
    }
  }
  const float part = lane < a.parts ? a.through[((int64_t)unit * chunks + c) * a.parts + lane] : 0.f;
  const float through = warp_sum(part);
  // rows from each token to its group's end, columns from the group's start to it
  float before[kG];
#pragma unroll
  for (int g = 0; g < kG; ++g) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float u = __shfl_down_sync(0xffffffffu, row[g], o), v = __shfl_up_sync(0xffffffffu, col[g], o);
      if (lane + o < 32) row[g] += u;
      if (lane >= o) col[g] += v;
    }
    before[g] = __shfl_up_sync(0xffffffffu, col[g], 1);
    if (lane == 0) before[g] = 0.f;
  }
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    float d = in[g] + row[g] + before[g] + through;
#pragma unroll
    for (int e = 0; e < kG; ++e) {
      if (e > g) d += __shfl_sync(0xffffffffu, row[e], 0);
      if (e < g) d += __shfl_sync(0xffffffffu, col[e], 31);
    }
    const int t = t0 + 32 * g + lane;
    if (t < end) a.d_lg[base + t] = d;
  }
}

template <typename T, int DA, bool GATE>
cudaError_t launch_pass(const DecayPass& a, const DecaySegs& g, int64_t blocks, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(decay_f32_kernel<T, DA, GATE>, sizeof(Smem<DA>), done);
  if (e != cudaSuccess) return e;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_pdl(decay_f32_kernel<T, DA, GATE>, dim3((unsigned)blocks), dim3(kThreads), sizeof(Smem<DA>), s, a, g);
}

template <typename T, int DA>
cudaError_t launch(const DecayPass& a, const DecaySegs& g, int64_t blocks, cudaStream_t s) {
  return a.x && !g.states_only ? launch_pass<T, DA, true>(a, g, blocks, s) : launch_pass<T, DA, false>(a, g, blocks, s);
}

cudaError_t dispatch(const DecayPass& a, lizard_dtype dt, const DecaySegs& g, int64_t blocks, cudaStream_t s) {
  if (dt == LIZARD_F32)
    return a.da == 64 ? launch<float, 64>(a, g, blocks, s) : launch<float, 128>(a, g, blocks, s);
  return a.da == 64 ? launch<bf16, 64>(a, g, blocks, s) : launch<bf16, 128>(a, g, blocks, s);
}

// One CTA an SM at da = 128, two at 64, by their shared memory; a state pass is a third of the work, a CTA's
// start and its state's way in and out two thirds of a chunk.
int f32_segments(int64_t ctas, int L, int da) {
  return decay_segments(ctas, da == 64 ? 304 : 152, (L + kC - 1) / kC, 0.35, 0.7, 0.4);
}

}  // namespace

int decay_segments(int64_t ctas, int per_wave, int chunks, double part, double start, double extra) {
  if (ctas >= 8 * per_wave) return 1;
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= 64 && s <= chunks; ++s) {
    const int cps = (chunks + s - 1) / s;
    if (s > 1 && (chunks + cps - 1) / cps < s) continue;  // some would be empty
    double t = (double)((ctas * s + per_wave - 1) / per_wave) * (cps + start);
    if (s > 1) t += part * (double)((ctas * (s - 1) + per_wave - 1) / per_wave) * (cps + start) + extra;
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

size_t decay_f32_workspace(int B, int H, int L, int da, int dc) {
  const int64_t ctas = (int64_t)B * H * (dc / kDc);
  return decay_seg_bytes(f32_segments(ctas, L, da), ctas, da);
}

cudaError_t launch_decay_f32(const DecayPass& a, lizard_dtype dt, float* ws, cudaStream_t s, int* launches) {
  const int64_t ctas = (int64_t)a.B * a.H * (a.dc / kDc);
  const int chunks = (a.L + kC - 1) / kC;
  DecaySegs g{};
  g.segs = f32_segments(ctas, a.L, a.da);
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
  trace_begin("decay_f32", s);
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
  const int64_t blocks = (int64_t)a.B * a.H * ((chunks + kGateWarps - 1) / kGateWarps);
  if (blocks > 0x7fffffffll || a.parts > 32) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(32 * kGateWarps);
  trace_begin("decay_gate", s);
  cudaError_t e = cudaErrorInvalidValue;
  if (a.in_slices == 1 && a.out_slices == 1) e = launch_pdl(decay_gate_kernel<1, 1>, grid, block, 0, s, a, chunks);
  if (a.in_slices == 1 && a.out_slices == 2) e = launch_pdl(decay_gate_kernel<1, 2>, grid, block, 0, s, a, chunks);
  if (a.in_slices == 2 && a.out_slices == 2) e = launch_pdl(decay_gate_kernel<2, 2>, grid, block, 0, s, a, chunks);
  if (a.in_slices == 1 && a.out_slices == 4) e = launch_pdl(decay_gate_kernel<1, 4>, grid, block, 0, s, a, chunks);
  trace_end(s);
  ++*launches;
  return e;
}

}  // namespace lz
