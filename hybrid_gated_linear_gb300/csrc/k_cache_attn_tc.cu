// k_cache_attn_tc.cu -- attention over the 8-bit paged cache for many new tokens per
// sequence (a chunk of a prompt), bf16, on tcgen05.
//
// Rows are the G = H / Hk query heads times the new tokens of a (sequence, key head), row =
// token * G + head.  One CTA takes 256 rows (two tiles of 128, the M of an MMA) and walks
// over the visible cache in blocks of 128 tokens:
//   3 warps   turn a block's codes into binary16 tiles (each code is exact in 11 bits); bulk
//             copies bring the codes into shared memory one block ahead (loads into registers
//             kept these warps waiting: 1.31 ms against 1.0 for 2 x 2048 tokens at 16384)
//   1 thread  issues S = Q K^T (operands in shared memory) and O += P V (P in tensor memory)
//   2 x 4 warps, one thread per row: running maxima and sum, P = 2^(z + e - mo) as binary16
//             over the columns S was read from
// The two tiles alternate, so the tensor cores work on one while the other's exponentials
// are taken.  z = logits in units of log 2, e = log2 of the page's value scale; m is the running
// maximum of z, for the sum, and mo, for the weights, that of z + e less kLift, whatever the
// pages' scales: binary16 holds 2^-24 to 2^16, and light tokens are lost at its low end.  O is
// rescaled only when the maximum has grown by more than kLazy.
//
// What bounds it: 4 D multiply-adds per row and token on the tensor cores against one
// exponential (32 per clock and SM) and a handful of fp32 operations per row and token; the
// cache's bytes are few.  One CTA per SM takes an equal share of the list of all blocks of
// all (sequence, rows, head), whatever their lengths; where a share ends inside one, its parts
// are joined by the last CTA to finish (fixed order: results do not depend on timing).
//
// Measured, H = 32, Hk = 8, D = 128, e4m3: two sequences, 2048 new tokens at 14336: 1.08 ms,
// 957 TFLOP/s (48% of the measured bf16 burst; bytes 1.23 ms, their conversion takes twice the
// operations; D = 64 0.95 ms, the same exponentials for half the products).  With the row warps' work left out 1.01, with the conversions left out 0.87, with
// both 0.64 ms: the roles contend for issue slots and shared memory, which the operands alone
// keep three quarters busy.  Staging the queries and joining parts cost about 80 us of it.
#include <algorithm>

#include "kv_cache.cuh"
#include "tc_pipe.cuh"

namespace lz {
namespace {

using namespace tc;

constexpr int kRows = 256;       // rows per CTA
constexpr int kBlock = 128;      // tokens per block
constexpr int kCodeWarps = 3;
constexpr int kMmaWarp = 8 + kCodeWarps;
// warps 0-7 rows, 8-10 codes, 11 MMA: twelve warps may have 168 registers per thread
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kMaxM = 16;
// Starting rows costs a CTA about as much as kCost blocks; pieces shorter than kMinBlocks are
// not worth joining.
constexpr int kCost = 6, kMinBlocks = 6;
// The weights' reference is set kLift below the running maximum, so P <= 2^(kLift + kLazy), a
// quarter of binary16's range: logits may be off by their own rounding.
constexpr float kLift = 6.f, kLazy = 8.f;
constexpr float kFar = 60.f;      // see weights()
constexpr float kLog2e = 1.4426950408889634f;

// Barriers: operand tiles full and free (two stages each), per row tile scores ready, weights
// written and output updated, scales of a block written (a ring of four); then the codes of
// keys and values in shared memory (RF, RF + 1) and read (RE, RE + 1).
enum { KF = 0, VF = 2, KE = 4, VE = 6, SF = 8, PF = 10, OD = 12, SC = 14, RF = 18, RE = 20, DONE = 22, NB = 23 };

template <int D>
struct Smem {
  static constexpr int kTile = kBlock * D * 2;
  static constexpr int Q = 0;                     // two tiles of 128 rows
  static constexpr int K = Q + 2 * kTile;         // two stages
  static constexpr int V = K + 2 * kTile;
  static constexpr int kRaw = kBlock * D;         // a block's codes
  static constexpr int R = V + 2 * kTile;         // of the keys, then of the values
  static constexpr int kBytes = R + 2 * kRaw;     // 224 KiB at D = 128
};

__device__ __forceinline__ uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D(tmem) (+)= A(tmem) * B(smem)^T ; issued by one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           bool accumulate) {
  const uint32_t acc = accumulate ? 1u : 0u;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Waits for the row's TMEM loads; the registers are named so that no use moves in front.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :
               : "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}

// A row's largest logit in each 16-token part of a block.  Checked: some token of the block
// may be hidden from the row, or a whole part unseen.
template <bool Checked>
__device__ __forceinline__ void part_maxima(uint32_t ts, const float2 (&sc)[8], float rs, int tok, int lo_r, int hi_r,
                                            float (&mb)[8]) {
  uint32_t u[2][32];
  tmem_ld32(ts, u[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    tmem_ld_wait32(u[q & 1]);
    if (q < 3) tmem_ld32(ts + 32 * (q + 1), u[(q + 1) & 1]);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float x = -INFINITY, y = -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        float s0 = __uint_as_float(u[q & 1][b * 16 + e]), s1 = __uint_as_float(u[q & 1][b * 16 + e + 1]);
        if (Checked) {
          const int c = tok + 32 * q + 16 * b + e;
          s0 = c >= lo_r && c <= hi_r ? s0 : -INFINITY;
          s1 = c + 1 >= lo_r && c + 1 <= hi_r ? s1 : -INFINITY;
        }
        x = fmaxf(x, s0), y = fmaxf(y, s1);
      }
      const float k = sc[2 * q + b].x;
      mb[2 * q + b] = !Checked || k > 0.f ? fmaxf(x, y) * (rs * k) : -INFINITY;
    }
  }
}

// Replaces a row's scores of a block by its weights 2^(z + e - mo) as binary16 and returns
// their sum in units of 2^m.  Checked additionally covers parts whose values are so much
// smaller than the others' that their weights would vanish before their share of the sum
// does: the sum then takes exponentials of its own.
template <bool Checked>
__device__ __forceinline__ float weights(uint32_t ts, const float2 (&sc)[8], float rs, int tok, int lo_r, int hi_r,
                                         float m, float mo) {
  float l = 0.f;
  uint32_t u[2][32];
  tmem_ld32(ts, u[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t pk[16];
    tmem_ld_wait32(u[q & 1]);
    if (q < 3) tmem_ld32(ts + 32 * (q + 1), u[(q + 1) & 1]);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float2 f = sc[2 * q + b];
      const float k = rs * f.x, sh = f.y - mo;
      float2 sum = make_float2(0.f, 0.f);
      float own = 0.f;
      const bool far = Checked && mo - f.y - m > kFar;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 x = make_float2(__uint_as_float(u[q & 1][b * 16 + e]), __uint_as_float(u[q & 1][b * 16 + e + 1]));
        float2 w;
        if (Checked) {
          const int c = tok + 32 * q + 16 * b + e;
          const float z0 = f.x > 0.f && c >= lo_r && c <= hi_r ? x.x * k : -INFINITY;
          const float z1 = f.x > 0.f && c + 1 >= lo_r && c + 1 <= hi_r ? x.y * k : -INFINITY;
          if (far) own += ex2_approx(z0 - m) + ex2_approx(z1 - m);
          w = make_float2(ex2_approx(z0 + sh), ex2_approx(z1 + sh));
        } else {
          const float2 z = f2_fma(x, make_float2(k, k), make_float2(sh, sh));
          w = make_float2(ex2_approx(z.x), ex2_approx(z.y));
        }
        sum = f2_add(sum, w);
        pk[b * 8 + e / 2] = half2_bits(w.x, w.y);
      }
      l += far ? own : (sum.x + sum.y) * ex2_approx(mo - f.y - m);
    }
    if (Checked) __syncwarp();
    // columns 16 q .. of the weights lie below the scores read so far and those in flight
    tmem_st16(ts + 16 * q, pk);
  }
  return l;
}

// What the rows of one (sequence, 256 rows) see; token numbers relative to base.  m counts
// them: sequence m / tiles, rows 256 (m % tiles) and on.
struct View {
  int64_t base, p0, first;
  int lo, hi;    // hi < lo: nothing
  int cnt, rows, r0;
  int units;     // blocks, at least one
};

__device__ __forceinline__ View view_of(const CacheAttn& a, int m, int tiles, int G) {
  View v;
  const int n = m / tiles;
  v.p0 = a.pos[n];
  v.cnt = a.count ? a.count[n] : a.T;
  v.first = a.first ? max((int64_t)0, a.first[n]) : 0;
  // rows of an unknown count are 0; with a bad position they see no cached token
  const bool known = v.cnt >= 0 && v.cnt <= a.T, placed = position_ok(v.p0);
  if (!known || !placed) raise_status(a.status, kDevCheck);
  v.cnt = known ? v.cnt : 0, v.p0 = placed ? v.p0 : 0;
  v.r0 = (m - n * tiles) * kRows;
  v.rows = max(0, min(kRows, v.cnt * G - v.r0));
  v.base = 0, v.lo = 0, v.hi = -1, v.units = 1;
  const int64_t all_lo = max(v.first, a.W > 0 ? v.p0 - a.W + 1 : (int64_t)0), all_hi = v.p0 + v.cnt - 1;
  if (placed && v.rows > 0 && all_lo <= all_hi) {
    if (!span_ok(a.c, all_lo, all_hi)) {
      raise_status(a.status, kDevCheck);
    } else {
      const int64_t lo = max(v.first, a.W > 0 ? v.p0 + v.r0 / G - a.W + 1 : (int64_t)0);
      const int64_t hi = v.p0 + (v.r0 + v.rows - 1) / G;
      if (lo <= hi) {
        v.base = lo & ~(int64_t)(kBlock - 1);
        v.lo = (int)(lo - v.base);
        v.hi = (int)(hi - v.base);
        v.units = v.hi / kBlock + 1;
      }
    }
  }
  return v;
}

// What the CTA works on: blocks ua .. ub-1 of one view and head, and where it is in the list.
struct Piece {
  View v;
  int64_t f, seg0;  // list indices: of the next piece, of view m's first entry (head 0)
  int m, n, hk, ua, ub;
  int c0, c1;       // the CTAs that share it
};

// The queries of a piece, rotated and scaled to a power of two near 2^13, as swizzled tiles; rs
// gets log2 e * scale * the power of two.  All warps.  Kept short on purpose: code that runs
// once per piece costs its instruction fetches.  Scratch: the rows' places, then the (cos, sin)
// pairs of the piece's tokens, in the key and value tiles.
template <int D>
__device__ __noinline__ void stage_queries(const CacheAttn& a, const Piece& s_p, unsigned char* tiles,
                                           float* s_rs, int64_t* s_off, int* s_tok, float2* s_cs) {
  constexpr int LPR = D / 4, RPI = 32 / LPR, WARPS = kThreads / 32;  // lanes per row, rows per step of a warp
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // every field once: through the references each use would be a load
  const RopeArgs rope = a.rope;
  const int G = a.H / a.c.Hk, rows = s_p.v.rows, r0 = s_p.v.r0, pairs = rope.rot / 2;
  const bf16* q0 = static_cast<const bf16*>(a.q) + s_p.n * a.sq.n;
  const float scale = a.scale * kLog2e;
  const int t0 = r0 / G;
  if (tid < kRows) {
    // rows beyond the call's point at the piece's first, which exists
    const int rr = r0 + tid < a.T * G ? r0 + tid : r0;
    const int tt = rr / G, h = s_p.hk * G + rr - tt * G;
    s_off[tid] = h * a.sq.h + tt * a.sq.t;
    s_tok[tid] = tt - t0;
  }
  if (rope.turns && rows > 0) {
    const int64_t p0 = s_p.v.p0 + t0;
    const int n = ((r0 + rows - 1) / G - t0 + 1) * pairs;
#pragma unroll 2
    for (int e = tid; e < n; e += kThreads) {
      const int t = e / pairs;
      float2 f;
      rope_angle(rope.turns[e - t * pairs], p0 + t, rope.factor, f.x, f.y);
      s_cs[e] = f;
    }
  }
  cta_sync();
  const int d0 = (lane % LPR) * 4;
  const bool half = rope.layout == LIZARD_ROPE_HALF, turn = rope.turns && d0 < rope.rot;
  // where the pairs' other channels are, if they lie together
  const int other = turn && half && pairs % 4 == 0 ? (d0 < pairs ? d0 + pairs : d0 - pairs) : d0;
  constexpr int RW = 4, RSTEP = RW * WARPS * RPI;
  // dead rows read row 0 (the loads stay free of branches, so all of them are in flight), and
  // the next rows' loads run ahead of this step's work
  Raw4<bf16> nx[RW], ny[RW];
  auto fetch = [&](int rb) {
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const int r = rb + k * WARPS * RPI + lane / LPR;
      const bf16* qp = q0 + s_off[r < rows ? r : 0];
      nx[k] = raw4(qp + d0);
      ny[k] = raw4(qp + other);
    }
  };
  fetch(warp * RPI);
#pragma unroll 1
  for (int rb = warp * RPI; rb < kRows; rb += RSTEP) {
    Raw4<bf16> x[RW], y[RW];
#pragma unroll
    for (int k = 0; k < RW; ++k) x[k] = nx[k], y[k] = ny[k];
    if (rb + RSTEP < kRows) fetch(rb + RSTEP);
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const int r = rb + k * WARPS * RPI + lane / LPR;
      const float4 xf = x[k].value(), yf = y[k].value();
      float v[4] = {xf.x, xf.y, xf.z, xf.w}, o[4] = {yf.x, yf.y, yf.z, yf.w};
      if (r >= rows) v[0] = v[1] = v[2] = v[3] = 0.f;
      if (turn && half && pairs % 4 != 0) {  // the pairs' other channels, one by one
        const bf16* qp = q0 + s_off[r < rows ? r : 0];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = d0 + i;
          o[i] = e < rope.rot ? ld_f(qp + (e < pairs ? e + pairs : e - pairs)) : 0.f;
        }
      } else if (!half) {
        o[0] = xf.y, o[1] = xf.x, o[2] = xf.w, o[3] = xf.z;
      }
      if (turn && half && pairs % 4 == 0) {
        const float s = d0 < pairs ? -1.f : 1.f;
        const float4* cs = reinterpret_cast<const float4*>(s_cs + s_tok[r < rows ? r : 0] * pairs +
                                                           (d0 < pairs ? d0 : d0 - pairs));
        const float4 f = cs[0], g = cs[1];
        v[0] = v[0] * f.x + s * o[0] * f.y, v[1] = v[1] * f.z + s * o[1] * f.w;
        v[2] = v[2] * g.x + s * o[2] * g.y, v[3] = v[3] * g.z + s * o[3] * g.w;
      } else if (turn && r < rows) {
        const float2* cs = s_cs + s_tok[r] * pairs;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = d0 + i;
          if (e < rope.rot) {
            const bool low = half ? e < pairs : (e & 1) == 0;
            const float2 f = cs[half ? (low ? e : e - pairs) : e >> 1];
            v[i] = v[i] * f.x + (low ? -o[i] : o[i]) * f.y;
          }
        }
      }
      float mx = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const int e = max(-126, min((int)(__float_as_uint(mx) >> 23) - 127 - 13, 113));
      const float inv = exp2_int(-e);
      if (r < kRows) {
        if (lane % LPR == 0) s_rs[r] = r < rows ? scale * exp2_int(e) : 1.f;
        *reinterpret_cast<uint2*>(tiles + (r >> 7) * (kBlock * D * 2) + sw128_offset(r & 127, d0, kBlock)) =
            make_uint2(half2_bits(v[0] * inv, v[1] * inv), half2_bits(v[2] * inv, v[3] * inv));
      }
    }
  }
  fence_proxy_async_smem();
}

// The partial results.  Formed where it is used: a pointer kept over a piece costs the row
// warps' loop spilled registers (2 x 2048 tokens at 14336: 1.12 ms against 1.08).
__device__ __forceinline__ float* parts_of(const CacheAttn& a) { return reinterpret_cast<float*>(a.ws + kCacheParts); }

// Where CTA c's partial result is: with the first block of its rows, or continuing them.
template <int D>
__device__ __forceinline__ size_t partial_at(int c, bool starts) {
  return (size_t)(2 * c + (starts ? 1 : 0)) * kRows * (D + 4);
}

// What the output functions read, copied once.
struct Out {
  const bf16 *q, *mk, *mv, *add;  // q, add, y at the piece's sequence
  bf16* y;
  int64_t qh, qt, ah, at, yh, yt;
  float scale, alpha;
  int G, M, TG, hk, r0, rows;
};
__device__ __forceinline__ Out out_of(const CacheAttn& a, const Piece& p) {
  Out o;
  o.q = static_cast<const bf16*>(a.q) + p.n * a.sq.n;
  o.mk = static_cast<const bf16*>(a.mk), o.mv = static_cast<const bf16*>(a.mv);
  o.add = a.add ? static_cast<const bf16*>(a.add) + p.n * a.sadd.n : nullptr;
  o.y = static_cast<bf16*>(a.y) + p.n * a.sy.n;
  o.qh = a.sq.h, o.qt = a.sq.t, o.ah = a.sadd.h, o.at = a.sadd.t, o.yh = a.sy.h, o.yt = a.sy.t;
  o.scale = a.scale * kLog2e, o.alpha = a.alpha;
  o.G = a.H / a.c.Hk, o.M = a.M, o.TG = a.T * o.G, o.hk = p.hk, o.r0 = p.v.r0, o.rows = p.v.rows;
  return o;
}

// Logits of the meta tokens of a row in units of log 2; they join its statistics.
template <int D>
__device__ __forceinline__ void with_meta(const Out& a, const bf16* q, int head, float (&zm)[kMaxM], float& m,
                                          float& l) {
  float top = m;
#pragma unroll
  for (int j = 0; j < kMaxM; ++j) {
    zm[j] = -INFINITY;
    if (j < a.M) {
      const bf16* k = a.mk + ((size_t)head * a.M + j) * D;
      float z = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 x = ld4(q + d), w = ld4(k + d);
        z += x.x * w.x + x.y * w.y + x.z * w.z + x.w * w.w;
      }
      zm[j] = z * a.scale;
      top = fmaxf(top, zm[j]);
    }
  }
  l = m == -INFINITY ? 0.f : l * exp2f(m - top);
#pragma unroll
  for (int j = 0; j < kMaxM; ++j)
    if (j < a.M) l += exp2f(zm[j] - top);
  m = top;
}

// Four channels of a row: o in units of 2^mo, normalised by (m, l), with the meta tokens' values
// and the other branch's output.
template <int D>
__device__ __forceinline__ float4 merged(const Out& a, float4 o, int head, int d, const float (&zm)[kMaxM],
                                         const bf16* add, float m, float mo, float l) {
  const float f = l > 0.f && mo != -INFINITY ? a.alpha / l * exp2f(mo - m) : 0.f;
  float4 v = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  if (a.M > 0) {
    const float fm = l > 0.f ? a.alpha / l : 0.f;
#pragma unroll
    for (int j = 0; j < kMaxM; ++j)
      if (j < a.M) {
        const float w = exp2f(zm[j] - m) * fm;
        const float4 x = ld4(a.mv + ((size_t)head * a.M + j) * D + d);
        v.x = fmaf(w, x.x, v.x), v.y = fmaf(w, x.y, v.y), v.z = fmaf(w, x.z, v.z), v.w = fmaf(w, x.w, v.w);
      }
  }
  if (add) {
    const float4 x = ld4(add + d);
    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
  }
  return v;
}

// A finished piece's rows, one thread per row (the first 256 threads): `to` is the thread's
// accumulator.
template <int D>
__device__ __noinline__ void write_rows(const CacheAttn& args, const Piece& p, uint32_t to, float m, float mo, float l) {
  const Out a = out_of(args, p);
  const int r = threadIdx.x, tt = (a.r0 + r) / a.G, head = a.hk * a.G + (a.r0 + r) % a.G;
  const bool live = r < a.rows, in_call = a.r0 + r < a.TG;
  bf16* y = a.y + head * a.yh + tt * a.yt;
  const bf16* add = a.add ? a.add + head * a.ah + tt * a.at : nullptr;
  float zm[kMaxM];
  if (live && a.M > 0) with_meta<D>(a, a.q + head * a.qh + tt * a.qt, head, zm, m, l);
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t u[16];
    __syncwarp();
    tmem_ld16(to + c, u);
    tmem_ld_wait();
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (live) {
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 o = merged<D>(a, make_float4(__uint_as_float(u[e]), __uint_as_float(u[e + 1]),
                                                  __uint_as_float(u[e + 2]), __uint_as_float(u[e + 3])),
                                   head, c + e, zm, add, m, mo, l);
        w[e / 2] = pack_bf16x2(o.x, o.y), w[e / 2 + 1] = pack_bf16x2(o.z, o.w);
      }
    }
    if (in_call) {
      *reinterpret_cast<uint4*>(y + c) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(y + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <int D>
__device__ __noinline__ void write_partial(float* mine, uint32_t to, float m, float mo, float l) {
  const int r = threadIdx.x;
  *reinterpret_cast<float4*>(mine + (size_t)kRows * D + 4 * r) = make_float4(m, mo, l, 0.f);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t u[32];
    tmem_ld32(to + c, u);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      *reinterpret_cast<uint4*>(mine + (size_t)r * D + c + e) = make_uint4(u[e], u[e + 1], u[e + 2], u[e + 3]);
  }
}

// The parts of CTAs c0 .. c1 joined.  First one thread per row merges the statistics (and the
// meta tokens'), then D / 4 lanes per row add the outputs, each part with its weight.  Scratch:
// per row the output maximum and the factor of the sum, then the meta tokens' weights.
template <int D>
__device__ __noinline__ void join_rows(const CacheAttn& args, const Piece& p, const float* part, float2* s_fin,
                                       float* s_meta, float* s_w) {
  constexpr int kKept = 32;  // parts whose weights fit the scratch
  constexpr int V4 = D / 4, STEP = kThreads / V4, RW = 4;
  const Out a = out_of(args, p);
  const int c0 = p.c0, c1 = p.c1, tid = threadIdx.x;
  if (tid < a.rows) {
    float m = -INFINITY, mo = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const float4 x =
          __ldcg(reinterpret_cast<const float4*>(part + partial_at<D>(c, c == c0) + (size_t)kRows * D + 4 * tid));
      const float mm = fmaxf(m, x.x);
      if (x.x != -INFINITY) l = (m == -INFINITY ? 0.f : l * exp2f(m - mm)) + x.z * exp2f(x.x - mm);
      m = mm, mo = fmaxf(mo, x.y);
    }
    float zm[kMaxM];
    if (a.M > 0) {
      const int tt = (a.r0 + tid) / a.G, head = a.hk * a.G + (a.r0 + tid) % a.G;
      with_meta<D>(a, a.q + head * a.qh + tt * a.qt, head, zm, m, l);
      const float f = l > 0.f ? a.alpha / l : 0.f;
#pragma unroll
      for (int j = 0; j < kMaxM; ++j)
        if (j < a.M) s_meta[tid * kMaxM + j] = exp2f(zm[j] - m) * f;
    }
    if (c1 - c0 < kKept)
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) {
        const float x = __ldcg(part + partial_at<D>(c, c == c0) + (size_t)kRows * D + 4 * tid + 1);
        s_w[(c - c0) * kRows + tid] = x == -INFINITY ? 0.f : exp2f(x - mo);
      }
    s_fin[tid] = make_float2(mo, l > 0.f && mo != -INFINITY ? a.alpha / l * exp2f(mo - m) : 0.f);
  }
  __syncthreads();
  const int k = tid % V4, d = 4 * k;
  // every lane of a warp takes every step: the shuffles need them
#pragma unroll 1
  for (int rb = 0; rb < kRows && a.r0 + rb < a.TG; rb += RW * STEP) {
    const int rl = rb + tid / V4;
    float4 v[RW];
#pragma unroll
    for (int q = 0; q < RW; ++q) v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int cb = c0; cb <= c1; cb += V4) {
      float wk[RW];  // of part cb + k
#pragma unroll
      for (int q = 0; q < RW; ++q) {
        const int r = rl + q * STEP;
        wk[q] = 0.f;
        if (c1 - c0 < kKept) {
          if (r < a.rows && cb + k <= c1) wk[q] = s_w[(cb + k - c0) * kRows + r];
        } else if (r < a.rows && cb + k <= c1) {
          const float mo = __ldcg(part + partial_at<D>(cb + k, cb + k == c0) + (size_t)kRows * D + 4 * r + 1);
          if (mo != -INFINITY) wk[q] = exp2f(mo - s_fin[r].x);
        }
      }
      const int cn = min(V4, c1 - cb + 1);
#pragma unroll 1
      for (int i = 0; i < cn; i += 2) {
        float4 o[RW][2];
#pragma unroll
        for (int q = 0; q < RW; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            o[q][e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (rl + q * STEP < a.rows && i + e < cn)
              o[q][e] = __ldcg(reinterpret_cast<const float4*>(part + partial_at<D>(cb + i + e, cb + i + e == c0) +
                                                               (size_t)(rl + q * STEP) * D + d));
          }
#pragma unroll
        for (int q = 0; q < RW; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w = __shfl_sync(0xffffffffu, wk[q], (i + e) & (V4 - 1), V4);
            v[q].x = fmaf(w, o[q][e].x, v[q].x), v[q].y = fmaf(w, o[q][e].y, v[q].y);
            v[q].z = fmaf(w, o[q][e].z, v[q].z), v[q].w = fmaf(w, o[q][e].w, v[q].w);
          }
      }
    }
#pragma unroll
    for (int q = 0; q < RW; ++q) {
      const int r = rl + q * STEP;
      if (r < kRows && a.r0 + r < a.TG) {
        const int tt = (a.r0 + r) / a.G, head = a.hk * a.G + (a.r0 + r) - tt * a.G;
        if (r < a.rows) {
          const float f = s_fin[r].y;
          v[q].x *= f, v[q].y *= f, v[q].z *= f, v[q].w *= f;
          for (int j = 0; j < a.M; ++j) {
            const float w = s_meta[r * kMaxM + j];
            const float4 x = ld4(a.mv + ((size_t)head * a.M + j) * D + d);
            v[q].x = fmaf(w, x.x, v[q].x), v[q].y = fmaf(w, x.y, v[q].y);
            v[q].z = fmaf(w, x.z, v[q].z), v[q].w = fmaf(w, x.w, v[q].w);
          }
          if (a.add) {
            const float4 x = ld4(a.add + head * a.ah + tt * a.at + d);
            v[q].x += x.x, v[q].y += x.y, v[q].z += x.z, v[q].w += x.w;
          }
        }
        st4(a.y + head * a.yh + tt * a.yt + d, v[q]);
      }
    }
    __syncwarp();
  }
}

template <int D, int F>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ CacheAttn a, int tiles) {
  using Sm = Smem<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ Ctl<NB> s_ctl;
  __shared__ float s_rs[kRows];
  // of a block's 16-token parts: key scale (0: unseen), log2 of the value scale
  __shared__ __align__(16) float2 s_scale[4][8];
  __shared__ int64_t s_sum[kThreads / 32];
  __shared__ Piece s_p;
  __shared__ int s_last;
  Ctl<NB>* ctl = &s_ctl;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.H / a.c.Hk, Hk = a.c.Hk;
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->bar[KF + i], kCodeWarps), mbar_init(&ctl->bar[VF + i], kCodeWarps);
      mbar_init(&ctl->bar[KE + i], 1), mbar_init(&ctl->bar[VE + i], 1);
      mbar_init(&ctl->bar[SF + i], 1), mbar_init(&ctl->bar[PF + i], 4), mbar_init(&ctl->bar[OD + i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&ctl->bar[SC + i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ctl->bar[RF + i], 1), mbar_init(&ctl->bar[RE + i], kCodeWarps);
    mbar_init(&ctl->bar[DONE], 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  pdl_wait();
  // How the blocks are shared out.  Either every view and head is cut into ceil(units / U) equal
  // pieces, U such that the pieces are at most as many as the CTAs; or the list of all blocks
  // (sequence-major, then rows, then head, kCost empty entries in front of each) is cut into equal
  // shares.  A CTA then has one piece, or several with a start and a join each: pieces are taken
  // while the longest is not longer than a share by more than those cost.
  const int M2 = a.c.N * tiles, segs = M2 * Hk, workers = gridDim.x;
  bool pieces = false;
  int64_t U = 1, share, f1;
  {
    __shared__ int s_most[kThreads / 32];
    const int mine = tid < M2 ? view_of(a, tid, tiles, G).units : 0;
    int64_t c = mine;
    int most = mine;
    for (int m = tid + kThreads; m < M2; m += kThreads) {
      const int u = view_of(a, m, tiles, G).units;
      c += u, most = max(most, u);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s_sum[warp] = c, s_most[warp] = most;
    __syncthreads();
    int64_t units = 0;
    for (int w = 0; w < kThreads / 32; ++w) units += s_sum[w], most = max(most, s_most[w]);
    units *= Hk;
    int64_t total = units + (int64_t)segs * kCost;
    share = max((total + workers - 1) / workers, (int64_t)(kMinBlocks + kCost));
    if (segs <= workers) {
      U = segs < workers ? min((units + workers - segs - 1) / (workers - segs), (int64_t)most) : most;
      U = max(U, (int64_t)kMinBlocks);
      int longest = 0;
      for (int m = tid; m < M2; m += kThreads) {
        const int u = m == tid ? mine : view_of(a, m, tiles, G).units;
        const int k = (int)((u + U - 1) / U);
        longest = max(longest, (u + k - 1) / k);
      }
      longest = __reduce_max_sync(0xffffffffu, longest);
      __syncthreads();
      if (lane == 0) s_most[warp] = longest;
      __syncthreads();
      for (int w = 0; w < kThreads / 32; ++w) longest = max(longest, s_most[w]);
      pieces = longest <= share + 2 * kCost;
    }
    if (pieces) share = 1, total = workers;
    const int64_t f = blockIdx.x * share;
    f1 = min(total, f + share);
    if (tid == 0) s_p.f = f1;  // nothing to do, unless found below
    int64_t before = 0;
    for (int m0 = 0; f < total && m0 < M2; m0 += kThreads) {
      const int m = m0 + tid;
      int64_t u = 0;
      if (m < M2) {
        const int n_u = m0 == 0 ? mine : view_of(a, m, tiles, G).units;
        u = Hk * (pieces ? (n_u + U - 1) / U : (int64_t)n_u + kCost);
      }
      c = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += x;
      }
      __syncthreads();
      if (lane == 31) s_sum[warp] = c;
      __syncthreads();
      for (int w = 0; w < warp; ++w) c += s_sum[w];
      c += before;
      if (f < c && f >= c - u) s_p.m = m, s_p.seg0 = c - u, s_p.f = f;
      for (int w = 0; w < kThreads / 32; ++w) before += s_sum[w];
      if (f < before) break;
    }
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  // one answer for the warp: what follows a wait is executed by all its lanes together
  auto wait_all = [&](int b, uint32_t parity) {
    const bool o = wait_bar(ctl, b, parity);
    return __all_sync(0xffffffffu, o) != 0;
  };
  int it = 0;  // blocks done in earlier pieces: stages and phases go on from there

  while (true) {
    if (tid == 0) {
      Piece& p = s_p;
      p.ub = 0;
      if (p.f < f1) {
        p.v = view_of(a, p.m, tiles, G);
        p.n = p.m / tiles;
        if (pieces) {
          const int k = (int)((p.v.units + U - 1) / U), i = (int)(p.f - p.seg0);
          p.hk = i / k;
          p.ua = (int)((int64_t)p.v.units * (i - p.hk * k) / k);
          p.ub = (int)((int64_t)p.v.units * (i - p.hk * k + 1) / k);
          p.c0 = (int)p.seg0 + p.hk * k;
          p.c1 = p.c0 + k - 1;
          p.f = f1;
        } else {
          const int entries = p.v.units + kCost;
          p.hk = (int)((p.f - p.seg0) / entries);
          const int64_t next = p.seg0 + (int64_t)(p.hk + 1) * entries, head0 = next - p.v.units;
          p.ua = (int)max((int64_t)0, p.f - head0);
          // 0: the share ends before this head's first block
          p.ub = (int)max((int64_t)0, min((int64_t)p.v.units, f1 - head0));
          p.c0 = (int)(head0 / share);
          p.c1 = (int)((next - 1) / share);
          p.f = next;
        }
        if (p.hk == Hk - 1) p.seg0 = p.f, ++p.m;
      }
    }
    cta_sync();
    if (s_p.ub == 0) break;
    const View& s_v = s_p.v;
    const int n = s_p.n, hk = s_p.hk, b0 = s_p.ua, nblk = s_p.ub - s_p.ua;
    const int rows = s_v.rows, r0 = s_v.r0;

    stage_queries<D>(a, s_p, sm + Sm::Q, s_rs, reinterpret_cast<int64_t*>(sm + Sm::R),
                     reinterpret_cast<int*>(sm + Sm::R) + 2 * kRows, reinterpret_cast<float2*>(sm + Sm::K));
    cta_sync();

    bool done_ok = true;
    float l = 0.f, m = -INFINITY, mo = -INFINITY;
    if (warp == kMmaWarp) {
      // ------------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        // descriptors differ in their address field (16-byte units) only: one addition per MMA,
        // since this thread's instructions are what the tensor cores wait for
        const uint32_t sb = smem_u32(sm);
        const uint64_t dq = desc_k(sb + Sm::Q, kBlock, 0), dk = desc_k(sb + Sm::K, kBlock, 0);
        const uint64_t dv = desc_mn(sb + Sm::V, kBlock, 0);
        constexpr uint32_t kTile16 = Sm::kTile / 16;
        const uint32_t id_s = idesc_f16(128, kBlock, false), id_o = idesc_f16(128, D, true);
        bool ok = true;
        auto scores = [&](int t, int i) {
          const uint64_t qa = dq + t * kTile16, kb = dk + (i & 1) * kTile16;  // i counts over all pieces
          const uint32_t ts = tmem + t * kBlock;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            constexpr uint32_t kCol = kBlock * 128 / 16;  // next 64 channels
            const uint32_t off = (j >> 2) * kCol + (j & 3) * 2;
            mma_bf16(ts, qa + off, kb + off, id_s, j > 0);
          }
          mma_commit(&ctl->bar[SF + t]);
          if (t == 1) mma_commit(&ctl->bar[KE + (i & 1)]);
        };
        const int end = it + nblk;
        if ((ok = wait_bar(ctl, KF + (it & 1), (it >> 1) & 1))) {
          tc_fence_after();
          scores(0, it), scores(1, it);
        }
        for (int i = it; ok && i < end; ++i) {
          const uint32_t par = (i >> 1) & 1;
          ok = wait_bar(ctl, VF + (i & 1), par);
          for (int t = 0; ok && t < 2; ++t) {
            if (!(ok = wait_bar(ctl, PF + t, i & 1))) break;
            tc_fence_after();
            const uint64_t vb = dv + (i & 1) * kTile16;
            const uint32_t to = tmem + 256 + t * D, ts = tmem + t * kBlock;
#pragma unroll
            for (int j = 0; j < kBlock / 16; ++j) mma_f16_ts(to, ts + 8 * j, vb + j * 128, id_o, j > 0 || i > it);
            mma_commit(&ctl->bar[OD + t]);
            if (t == 1) mma_commit(&ctl->bar[VE + (i & 1)]);
            if (i + 1 < end) {
              if (t == 0 && !(ok = wait_bar(ctl, KF + ((i + 1) & 1), ((i + 1) >> 1) & 1))) break;
              tc_fence_after();
              scores(t, i + 1);
            }
          }
        }
        if (!ok) ctl->abort = 1;
      }
    } else if (warp >= 8) {
      // ------------------------------------------------------------------ codes -> binary16
      // Warp w takes the 16-token parts w, w + 3, w + 6 of a block: IT steps of 32 chunks each.
      constexpr int IT = D / 32, NP = (8 + kCodeWarps - 1) / kCodeWarps;
      const int w = warp - 8;
      // Eight lanes that access together hold four chunks each of two rows.  At D = 128 the rows
      // are r and r ^ 5: the codes they read lie in different halves of the banks (chunk c of row r
      // is at place c ^ (r & 7)), and so do the binary16 chunks they store, 2 c ^ (r & 7).
      const int chunk = D == 128 ? 4 * ((lane >> 3) & 1) + (lane & 3) : lane & 3;
      const int row = D == 128 ? ((lane >> 4) & 1) ^ ((lane & 4) ? 5 : 0) : lane >> 2;
      auto row_of = [&](int k) { return D == 128 ? 8 * (k >> 1) + (row ^ (2 * (k & 1))) : 8 * k + row; };
      const int lo = s_v.lo, hi = s_v.hi;
      const int64_t base = s_v.base;
      // Four blocks are looked up at a time: lane 8 b + p has part p of block b.  The page numbers
      // of the batch after next are on their way while the next batch's scales are.
      int at = -1, nat = -1;  // where the part is (in parts of 16 rows; -1: unseen)
      uint32_t full = 0, nfull = 0;  // the lanes whose part exists
      float2 sc = make_float2(0.f, 0.f), nsc = sc;
      int id = -1;
      auto token = [&](int i) { return (b0 + i + (lane >> 3)) * kBlock + (lane & 7) * 16; };
      auto look = [&](int i) {
        id = -2;  // nothing to see
        const int tok = token(i);
        if (i + (lane >> 3) < nblk && tok + 15 >= lo && tok <= hi)
          id = a.c.table[(size_t)n * a.c.max_pages + (uint32_t)((base + tok) >> a.c.log_p) % (uint32_t)a.c.max_pages];
      };
      auto find = [&](int i) {
        nat = -1;
        nsc = make_float2(0.f, 0.f);
        if ((unsigned)id < (unsigned)a.c.pages) {
          const size_t ph = (size_t)id * Hk + hk;
          nat = (int)((ph * a.c.P + (int)((base + token(i)) & (a.c.P - 1))) >> 4);
          nsc = make_float2(a.c.ks[ph], a.c.vs[ph]);
        } else if (id != -2) {
          raise_status(a.status, kDevCheck);
        }
        nfull = __ballot_sync(0xffffffffu, nat >= 0);
      };
      // Copies block i's codes (x = 0 keys, 1 values); past the batch in `at`, it is the next one's.
      auto copy = [&](int x, int i) {
        const uint32_t mask = ((i & 3) ? full : nfull) >> ((i & 3) * 8) & 0xff;
        const int part = __shfl_sync(0xffffffffu, (i & 3) ? at : nat, (i & 3) * 8 + (lane & 7));
        if (lane == 0) mbar_arrive_expect_tx(&ctl->bar[RF + x], __popc(mask) * 16 * D);
        __syncwarp();
        if (lane < 8 && part >= 0)
          bulk_load(sm + Sm::R + x * Sm::kRaw + lane * 16 * D, (x ? a.c.v : a.c.k) + (size_t)part * (16 * D), 16 * D,
                    &ctl->bar[RF + x]);
      };
      auto convert = [&](const unsigned char* raw, unsigned char* tile, int i) {
        const int tok = (b0 + i) * kBlock;
        const uint32_t mask = full >> ((i & 3) * 8) & 0xff;
        // parts that end beyond what is seen hold bytes that were never written
        const bool whole = mask == 0xff && tok >= lo && tok + kBlock - 1 <= hi;
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          const int p = w + q * kCodeWarps;
          if (p >= 8) break;
          uint4 u[IT];
#pragma unroll
          for (int k = 0; k < IT; ++k) {
            const int r = row_of(k);
            u[k] = *reinterpret_cast<const uint4*>(raw + (p * 16 + r) * D + 16 * chunk_place<D>(r, chunk));
          }
          if (!whole) {
#pragma unroll
            for (int k = 0; k < IT; ++k) {
              const int tk = tok + 16 * p + row_of(k);
              if (!(mask >> p & 1) || tk < lo || tk > hi) u[k] = make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int k = 0; k < IT; ++k) {
            const int r = row_of(k);
            uint32_t h[8];
            const uint32_t x[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) codes_to_half<F>(x[e], h[2 * e], h[2 * e + 1]);
            unsigned char* t = tile + p * 16 * 128;
            *reinterpret_cast<uint4*>(t + sw128_offset(r, 16 * chunk, kBlock)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(t + sw128_offset(r, 16 * chunk + 8, kBlock)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
        }
        fence_proxy_async_smem();
      };
      look(0);
      find(0);
      look(4);
      if (w < 2) copy(w, 0);
      bool ok = true;
      for (int i = 0; i < nblk; ++i) {
        const int gi = it + i, st = gi & 1;  // gi counts over all pieces
        const uint32_t free_par = ((gi >> 1) & 1) ^ 1;
        if ((i & 3) == 0) {
          at = nat, sc = nsc, full = nfull;
          find(i + 4);
          look(i + 8);
        }
        // Keys, then values.  Warp x copies the next block's once all three have read this one's.
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          if (gi >= 2 && !(ok = wait_all((x ? VE : KE) + st, free_par))) break;
          if (x == 0 && w == 0) {
            // Block i - 4's scales are no longer read: the keys' stage is free, so the scores of
            // block i - 2 are done, which were issued after every row had finished block i - 3.
            if (lane >> 3 == (i & 3))
              s_scale[gi & 3][lane & 7] =
                  make_float2(sc.x, at >= 0 ? (float)((int)(__float_as_uint(sc.y) >> 23 & 0xff) - 127) : 0.f);
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->bar[SC + (gi & 3)]);
          }
          if (!(ok = wait_all(RF + x, gi & 1))) break;
          convert(sm + Sm::R + x * Sm::kRaw, sm + (x ? Sm::V : Sm::K) + st * Sm::kTile, i);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->bar[(x ? VF : KF) + st]), mbar_arrive(&ctl->bar[RE + x]);
          if (w == x && i + 1 < nblk) {
            if (!(ok = wait_all(RE + x, gi & 1))) break;
            copy(x, i + 1);
          }
        }
        if (!ok) break;
      }
      if (!ok) ctl->abort = 1;
    } else {
      // ------------------------------------------------------------------ rows
      const int t = warp >> 2, r = warp * 32 + lane;  // row tile, row of the CTA
      const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t ts = tl + t * kBlock, to = tl + 256 + t * D;
      const float rs = s_rs[r];
      auto sees_from = [&](int64_t p) {
        const int64_t x = max(s_v.first, a.W > 0 ? p - a.W + 1 : (int64_t)0) - s_v.base;
        return (int)max((int64_t)0, min(x, (int64_t)0x7fffffff));
      };
      const int64_t p = s_v.p0 + (r0 + r) / G;
      const int lo_r = sees_from(p), hi_r = r < rows ? (int)(p - s_v.base) : -1;
      // tokens every live row of the tile sees (dead rows may see anything)
      const int last = min(rows, 128 * t + 128) - 1;
      const int all_lo = last >= 128 * t ? sees_from(s_v.p0 + (r0 + last) / G) : 0;
      const int all_hi = last >= 128 * t ? (int)(s_v.p0 + (r0 + 128 * t) / G - s_v.base) : 0x7fffffff;
      bool ok = true;
      for (int i = 0; i < nblk; ++i) {
        const int tok = (b0 + i) * kBlock;
        const int gi = it + i;  // counts over all pieces
        if (!(ok = wait_all(SC + (gi & 3), (gi >> 2) & 1) && wait_all(SF + t, gi & 1))) break;
        tc_fence_after();
        float2 sc[8];
#pragma unroll
        for (int b = 0; b < 8; b += 2) {
          const float4 x = *reinterpret_cast<const float4*>(&s_scale[gi & 3][b]);
          sc[b] = make_float2(x.x, x.y), sc[b + 1] = make_float2(x.z, x.w);
        }
        bool checked = tok < all_lo || tok + kBlock - 1 > all_hi;
#pragma unroll
        for (int b = 0; b < 8; ++b) checked |= sc[b].x == 0.f;
        float mb[8], mn = m, top = -INFINITY;
        if (checked) part_maxima<true>(ts, sc, rs, tok, lo_r, hi_r, mb);
        else part_maxima<false>(ts, sc, rs, tok, lo_r, hi_r, mb);
#pragma unroll
        for (int b = 0; b < 8; ++b) mn = fmaxf(mn, mb[b]), top = fmaxf(top, mb[b] + sc[b].y);
        const float mon = fmaxf(mo, top - kLift);
        // the sum's scale follows m exactly, the output's only in steps
        if (mn > m) l *= exp2f(m - mn), m = mn;
        const bool jump = mon > mo + kLazy;
        if (__any_sync(0xffffffffu, jump)) {
          const float f = mon > mo ? exp2f(mo - mon) : 1.f;
          mo = fmaxf(mo, mon);
          if (i > 0) {
            if (!(ok = wait_all(OD + t, (gi - 1) & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t u[32];
              tmem_ld32(to + c, u);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * f);
              tmem_st32(to + c, u);
            }
            tmem_st_wait();
          }
        }
        const float ml = m == -INFINITY ? 0.f : m, mol = mo == -INFINITY ? 0.f : mo;
        bool far = false;
#pragma unroll
        for (int b = 0; b < 8; ++b) far |= mol - sc[b].y - ml > kFar;
        if (__any_sync(0xffffffffu, checked || far)) l += weights<true>(ts, sc, rs, tok, lo_r, hi_r, ml, mol);
        else l += weights<false>(ts, sc, rs, tok, lo_r, hi_r, ml, mol);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->bar[PF + t]);
      }
      if (ok && (ok = wait_all(OD + t, (it + nblk - 1) & 1))) tc_fence_after();
      if (!ok) ctl->abort = 1;
      done_ok = ok;
    }

    // ---- output
    const bool alone = s_p.ua == 0 && s_p.ub == s_v.units;
    if (warp < 8 && __all_sync(0xffffffffu, done_ok && !*(volatile int*)&ctl->abort)) {
      const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 + (warp >> 2) * D;
      if (alone) write_rows<D>(a, s_p, to, m, mo, l);
      else write_partial<D>(parts_of(a) + partial_at<D>(blockIdx.x, s_p.ua == 0), to, m, mo, l);
    }
    it += nblk;
    tc_fence_before();
    cta_sync();
    tc_fence_after();
    if (*(volatile int*)&ctl->abort) break;
    if (!alone) {
      __threadfence();
      __syncthreads();
      const int c0 = s_p.c0, c1 = s_p.c1;
      unsigned* counter = reinterpret_cast<unsigned*>(a.ws) + c0;
      if (tid == 0) s_last = atomicAdd(counter, 1u) == (unsigned)(c1 - c0);
      __syncthreads();
      if (s_last) {
        __threadfence();
        join_rows<D>(a, s_p, parts_of(a), reinterpret_cast<float2*>(sm + Sm::K),
                     reinterpret_cast<float*>(sm + Sm::V), reinterpret_cast<float*>(sm + Sm::Q));
        if (tid == 0) *counter = 0u;
      }
    }
    cta_sync();  // before s_p and the queries' tiles are written again
  }
  if (warp == kMmaWarp) {
    if (lane == 0) {
      mma_commit(&ctl->bar[DONE]);
      drain_bar(ctl, DONE, 1, globaltimer_ns());
    }
    __syncwarp();
  }
  tc_fence_before();
  cta_sync();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (*(volatile int*)&ctl->abort) {
    if (tid == 0) raise_status(a.status, kDevTimeout);
    // a wait gave up after a second; copies issued just before the others saw that land well
    // within a millisecond
    const long long c0 = clock64();
    while (clock64() - c0 < 4000000ll) {
    }
  }
  pdl_trigger();
}

constexpr int kMaxCtas = 152;  // one per SM; sizes the scratch

template <int D, int F>
cudaError_t launch(const CacheAttn& a, cudaStream_t s, int* launches) {
  const int tiles = (a.H / a.c.Hk * a.T + kRows - 1) / kRows;
  constexpr int smem = Smem<D>::kBytes + 1024;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(prompt_kernel<D, F>, smem, done);
  if (e != cudaSuccess) return e;
  trace_begin("cache_attn_prompt", s);
  e = launch_pdl(prompt_kernel<D, F>, dim3(std::min(ctas_per_wave(1), kMaxCtas)), dim3(kThreads), smem, s, a, tiles);
  trace_end(s);
  ++*launches;
  return e;
}

}  // namespace

// Us for H = 32, Hk = 8, d = 128, here against k_cache_attn.cu with as many rows: 128 rows 137
// against 272 (eight sequences of 8192 tokens), 145 against 285 (one of 65536), 53 against 58 (one
// of 1000), 34 against 63 (eight of 200); 64 rows 134 against 130, 136 against 143, 46 against 34,
// 33 against 29; 32 rows 130 against 72 (eight of 8192).
bool cache_attn_tc_used(int H, int Hk, int T, lizard_dtype dt) { return dt == LIZARD_BF16 && H / Hk * T > 64; }

size_t cache_attn_tc_workspace(int d) {
  // the counters, then two partial results per CTA
  return kCacheParts + (size_t)2 * kMaxCtas * kRows * (d + 4) * sizeof(float);
}

cudaError_t launch_cache_attn_tc(const CacheAttn& a, cudaStream_t s, int* launches) {
  if (a.c.d == 64)
    return a.c.fmt == LIZARD_KV_E4M3 ? launch<64, 0>(a, s, launches) : launch<64, 1>(a, s, launches);
  return a.c.fmt == LIZARD_KV_E4M3 ? launch<128, 0>(a, s, launches) : launch<128, 1>(a, s, launches);
}

}  // namespace lz
