// k_cache_attn_tc.cu -- attention over the 8-bit paged cache for many new tokens per
// sequence (a chunk of a prompt), bf16, on tcgen05.
//
// Rows are the G = H / Hk query heads times the new tokens of a (sequence, key head), row =
// token * G + head.  One CTA takes 256 rows (two tiles of 128, the M of an MMA) and walks
// over the visible cache in blocks of 128 tokens:
//   3 warps   turn a block's codes into binary16 tiles (each code is exact in 11 bits); the
//             copy from global memory runs one block ahead in registers
//   1 thread  issues S = Q K^T (operands in shared memory) and O += P V (P in tensor memory)
//   2 x 4 warps, one thread per row: running maxima and sum, P = 2^(z + e - mo) as binary16
//             over the columns S was read from
// The two tiles alternate, so the tensor cores work on one while the other's exponentials
// are taken.  z = logits in units of log 2, e = log2 of the page's value scale; mo is the
// running maximum of z + e, so the weights stay near (0, 1] whatever the pages' scales, and
// m that of z, for the sum.  O is rescaled only when mo has grown by more than 2^kLazy.
//
// What bounds it: 4 D multiply-adds per row and token on the tensor cores against one
// exponential (32 per clock and SM) and a handful of fp32 operations per row and token; the
// cache's bytes are few.  When there are fewer CTAs than SMs, each CTA's cache range is cut
// into pieces, joined by the last CTA to finish (fixed order).
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
constexpr float kLazy = 8.f;     // P <= 2^8 fits binary16 with room for its sums
constexpr float kFar = 60.f;      // see weights()
constexpr float kLog2e = 1.4426950408889634f;

// Barriers: operand tiles full and free (two stages each), per row tile scores ready, weights
// written and output updated, scales of a block written (a ring of four).
enum { KF = 0, VF = 2, KE = 4, VE = 6, SF = 8, PF = 10, OD = 12, SC = 14, DONE = 18, NB = 19 };

template <int D>
struct Smem {
  static constexpr int kTile = kBlock * D * 2;
  static constexpr int Q = 0;                     // two tiles of 128 rows
  static constexpr int K = Q + 2 * kTile;         // two stages
  static constexpr int V = K + 2 * kTile;
  static constexpr int kBytes = V + 2 * kTile;    // 192 KiB at D = 128
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

// Two fp32 multiply-adds or additions in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
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
          const float2 z = fma2(x, make_float2(k, k), make_float2(sh, sh));
          w = make_float2(ex2_approx(z.x), ex2_approx(z.y));
        }
        sum = add2(sum, w);
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

// What this CTA's rows see; token numbers relative to base.
struct View {
  int64_t base, p0, first;
  int lo, hi, cnt, rows, r0;
  int b0, b1;  // its blocks
};

template <int D, int F>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(CacheAttn a, int tiles, int splits) {
  using Sm = Smem<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ Ctl<NB> s_ctl;
  __shared__ float s_rs[kRows];
  __shared__ __align__(16) float2 s_scale[4][8];  // of a block's 16-token parts: key scale (0: unseen), log2 of the value scale
  __shared__ View s_v;
  __shared__ int s_last;
  Ctl<NB>* ctl = &s_ctl;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.H / a.c.Hk, Hk = a.c.Hk;
  // the tiles with the most to see first
  const int split = blockIdx.x % splits, unit = blockIdx.x / splits;
  const int nh = unit % (a.c.N * Hk), tile = tiles - 1 - unit / (a.c.N * Hk);
  const int n = nh / Hk, hk = nh % Hk;

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
    mbar_init(&ctl->bar[DONE], 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (tid == 0) {
    View v;
    v.p0 = a.pos[n];
    v.cnt = a.count ? a.count[n] : a.T;
    v.first = a.first ? max((int64_t)0, a.first[n]) : 0;
    const bool known = v.cnt >= 0 && v.cnt <= a.T && v.p0 >= 0;
    if (!known) raise_status(a.status, kDevCheck);
    v.cnt = known ? v.cnt : 0;
    v.r0 = tile * kRows;
    v.rows = max(0, min(kRows, v.cnt * G - v.r0));
    v.base = 0, v.lo = 0, v.hi = -1;
    const int64_t all_lo = max(v.first, a.W > 0 ? v.p0 - a.W + 1 : (int64_t)0), all_hi = v.p0 + v.cnt - 1;
    if (v.rows > 0 && all_lo <= all_hi) {
      if (!span_ok(a.c, all_lo, all_hi)) {
        raise_status(a.status, kDevCheck);
      } else {
        const int64_t lo = max(v.first, a.W > 0 ? v.p0 + v.r0 / G - a.W + 1 : (int64_t)0);
        const int64_t hi = v.p0 + (v.r0 + v.rows - 1) / G;
        if (lo <= hi) {
          v.base = lo & ~(int64_t)(kBlock - 1);
          v.lo = (int)(lo - v.base);
          v.hi = (int)(hi - v.base);
        }
      }
    }
    const int nb = v.hi < v.lo ? 0 : v.hi / kBlock + 1;
    v.b0 = (int)((int64_t)nb * split / splits);
    v.b1 = (int)((int64_t)nb * (split + 1) / splits);
    s_v = v;
  }
  cta_sync();
  const int rows = s_v.rows, r0 = s_v.r0, nblk = s_v.b1 - s_v.b0;

  // ---- queries: rotated, scaled to a power of two near 2^13, as swizzled tiles
  if (warp < 8) {
    constexpr int LPR = D / 4, RPI = 32 / LPR;  // lanes per row, rows per step of a warp
    const int d0 = (lane % LPR) * 4, hr = a.rope.rot / 2;
    const bool half = a.rope.layout == LIZARD_ROPE_HALF;
    float co[4], si[4];
    int angle_of = -1;  // token whose angles co, si hold
    for (int k0 = 0; k0 < 32; k0 += 4 * RPI) {
      float x[4][4], y[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = warp * 32 + k0 + k * RPI + lane / LPR;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f), o = v;
        if (r < rows) {
          const int tt = (r0 + r) / G, h = hk * G + (r0 + r) % G;
          const bf16* qp = static_cast<const bf16*>(a.q) + n * a.sq.n + h * a.sq.h + tt * a.sq.t;
          v = ld4(qp + d0);
          if (a.rope.turns && half && d0 < a.rope.rot) {
            auto other = [&](int e) { return e < a.rope.rot ? ld_f(qp + (e < hr ? e + hr : e - hr)) : 0.f; };
            if (hr % 4 == 0) o = ld4(qp + (d0 < hr ? d0 + hr : d0 - hr));
            else o = make_float4(other(d0), other(d0 + 1), other(d0 + 2), other(d0 + 3));
          } else {
            o = make_float4(v.y, v.x, v.w, v.z);
          }
        }
        x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
        y[k][0] = o.x, y[k][1] = o.y, y[k][2] = o.z, y[k][3] = o.w;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = warp * 32 + k0 + k * RPI + lane / LPR;
        float v[4] = {x[k][0], x[k][1], x[k][2], x[k][3]};
        if (a.rope.turns && r < rows && d0 < a.rope.rot) {
          const int tt = (r0 + r) / G;
          if (tt != angle_of) {
            angle_of = tt;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int e = d0 + i;
              float c = 1.f, s = 0.f;
              if (e < a.rope.rot) {
                const bool low = half ? e < hr : (e & 1) == 0;
                rope_angle(a.rope.turns[half ? (low ? e : e - hr) : e >> 1], s_v.p0 + tt, a.rope.factor, c, s);
                if (low) s = -s;
              }
              if (i == 0) co[0] = c, si[0] = s;
              else if (i == 1) co[1] = c, si[1] = s;
              else if (i == 2) co[2] = c, si[2] = s;
              else co[3] = c, si[3] = s;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = v[i] * co[i] + y[k][i] * si[i];
        }
        float mx = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        int e = (int)(__float_as_uint(mx) >> 23) - 127 - 13;
        e = max(-126, min(e, 113));
        const float inv = exp2_int(-e);
        if (lane % LPR == 0) s_rs[r] = r < rows ? a.scale * kLog2e * exp2_int(e) : 1.f;
        *reinterpret_cast<uint2*>(sm + Sm::Q + (r >> 7) * Sm::kTile + sw128_offset(r & 127, d0, kBlock)) =
            make_uint2(half2_bits(v[0] * inv, v[1] * inv), half2_bits(v[2] * inv, v[3] * inv));
      }
    }
    fence_proxy_async_smem();
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
        const uint64_t qa = dq + t * kTile16, kb = dk + (i & 1) * kTile16;
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
      if (nblk > 0 && (ok = wait_bar(ctl, KF, 0))) {
        tc_fence_after();
        scores(0, 0), scores(1, 0);
      }
      for (int i = 0; ok && i < nblk; ++i) {
        const uint32_t par = (i >> 1) & 1;
        ok = wait_bar(ctl, VF + (i & 1), par);
        for (int t = 0; ok && t < 2; ++t) {
          if (!(ok = wait_bar(ctl, PF + t, i & 1))) break;
          tc_fence_after();
          const uint64_t vb = dv + (i & 1) * kTile16;
          const uint32_t to = tmem + 256 + t * D, ts = tmem + t * kBlock;
#pragma unroll
          for (int j = 0; j < kBlock / 16; ++j) mma_f16_ts(to, ts + 8 * j, vb + j * 128, id_o, j > 0 || i > 0);
          mma_commit(&ctl->bar[OD + t]);
          if (t == 1) mma_commit(&ctl->bar[VE + (i & 1)]);
          if (i + 1 < nblk) {
            if (t == 0 && !(ok = wait_bar(ctl, KF + ((i + 1) & 1), ((i + 1) >> 1) & 1))) break;
            tc_fence_after();
            scores(t, i + 1);
          }
        }
      }
      if (!ok) ctl->abort = 1;
      mma_commit(&ctl->bar[DONE]);
      drain_bar(ctl, DONE, 1, globaltimer_ns());
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ codes -> binary16
    // Warp w takes the 16-token parts w, w + 3, w + 6 of a block: IT steps of 32 chunks each.
    constexpr int IT = D / 32, RPS = 16 / IT, NP = (8 + kCodeWarps - 1) / kCodeWarps;
    const int w = warp - 8;
    // Eight lanes that store together hold half rows (64 channels) of two rows: their stores
    // fall into different banks.  A step adds 4 (8) rows.
    const int row = D == 128 ? 2 * (lane >> 4) + ((lane >> 2) & 1) : lane >> 2;
    const int chunk = D == 128 ? 4 * ((lane >> 3) & 1) + (lane & 3) : lane & 3;
    const int lo = s_v.lo, hi = s_v.hi;
    const int64_t base = s_v.base;
    // Four blocks are looked up at a time, the next four while these are converted: lane
    // 8 b + p has part p of block b, where it is (in parts of 16 rows) and its scales.
    int at = -1, nat = -1;
    float2 sc = make_float2(0.f, 0.f), nsc = sc;
    auto look = [&](int i) {
      i += lane >> 3;
      nat = -1;
      nsc = make_float2(0.f, 0.f);
      const int tok = (s_v.b0 + i) * kBlock + (lane & 7) * 16;
      if (i < nblk && tok + 15 >= lo && tok <= hi) {
        const int id = pool_page(a.c, n, (uint32_t)((base + tok) >> a.c.log_p));
        if (id < 0) {
          raise_status(a.status, kDevCheck);
        } else {
          const size_t ph = (size_t)id * Hk + hk;
          nat = (int)((ph * a.c.P + (int)((base + tok) & (a.c.P - 1))) >> 4);
          nsc = make_float2(a.c.ks[ph], (float)((int)(__float_as_uint(a.c.vs[ph]) >> 23 & 0xff) - 127));
        }
      }
    };
    auto load = [&](const unsigned char* pool, int i, uint4 (&u)[NP][IT]) {
      const int tok = (s_v.b0 + i) * kBlock;
      // parts that end beyond what is seen hold bytes that were never written
      const bool inner = tok >= lo && tok + kBlock - 1 <= hi;
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const int p = w + q * kCodeWarps;
        // past the batch in `at`, block i is the first of the next one
        const int part = __shfl_sync(0xffffffffu, (i & 3) ? at : nat, (i & 3) * 8 + (p & 7));
        const unsigned char* src = pool + (size_t)part * (16 * D);
#pragma unroll
        for (int k = 0; k < IT; ++k) {
          const int r = row + k * RPS, tk = tok + 16 * p + r;
          u[q][k] = make_uint4(0, 0, 0, 0);
          if (p < 8 && i < nblk && part >= 0 && (inner || (tk >= lo && tk <= hi)))
            u[q][k] = *reinterpret_cast<const uint4*>(src + r * D + 16 * chunk_place<D>(r, chunk));
        }
      }
    };
    auto convert = [&](unsigned char* tile, const uint4 (&u)[NP][IT]) {
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const int p = w + q * kCodeWarps;
        if (p >= 8) break;
#pragma unroll
        for (int k = 0; k < IT; ++k) {
          const int r = row + k * RPS;
          uint32_t h[8];
          const uint32_t x[4] = {u[q][k].x, u[q][k].y, u[q][k].z, u[q][k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) codes_to_half<F>(x[e], h[2 * e], h[2 * e + 1]);
          unsigned char* t = tile + p * 16 * 128;
          *reinterpret_cast<uint4*>(t + sw128_offset(r, 16 * chunk, kBlock)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(t + sw128_offset(r, 16 * chunk + 8, kBlock)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      }
      fence_proxy_async_smem();
    };
    uint4 ku[NP][IT], vu[NP][IT];
    look(0);
    load(a.c.k, 0, ku);
    load(a.c.v, 0, vu);
    bool ok = true;
    for (int i = 0; i < nblk; ++i) {
      const int st = i & 1;
      const uint32_t free_par = ((i >> 1) & 1) ^ 1;
      if ((i & 3) == 0) {
        at = nat, sc = nsc;
        look(i + 4);
      }
      if (i >= 2 && !(ok = wait_all(KE + st, free_par))) break;
      // Block i - 4's scales are no longer read: the keys' stage is free, so the scores of block
      // i - 2 are done, which were issued after every row had finished block i - 3.
      if (w == 0) {
        if (lane >> 3 == (i & 3)) s_scale[i & 3][lane & 7] = sc;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->bar[SC + (i & 3)]);
      }
      convert(sm + Sm::K + st * Sm::kTile, ku);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[KF + st]);
      load(a.c.k, i + 1, ku);
      if (i >= 2 && !(ok = wait_all(VE + st, free_par))) break;
      convert(sm + Sm::V + st * Sm::kTile, vu);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[VF + st]);
      load(a.c.v, i + 1, vu);
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
      const int tok = (s_v.b0 + i) * kBlock;
      if (!(ok = wait_all(SC + (i & 3), (i >> 2) & 1) && wait_all(SF + t, i & 1))) break;
      tc_fence_after();
      float2 sc[8];
#pragma unroll
      for (int b = 0; b < 8; b += 2) {
        const float4 x = *reinterpret_cast<const float4*>(&s_scale[i & 3][b]);
        sc[b] = make_float2(x.x, x.y), sc[b + 1] = make_float2(x.z, x.w);
      }
      bool checked = tok < all_lo || tok + kBlock - 1 > all_hi;
#pragma unroll
      for (int b = 0; b < 8; ++b) checked |= sc[b].x == 0.f;
      float mb[8], mn = m, mon = mo;
      if (checked) part_maxima<true>(ts, sc, rs, tok, lo_r, hi_r, mb);
      else part_maxima<false>(ts, sc, rs, tok, lo_r, hi_r, mb);
#pragma unroll
      for (int b = 0; b < 8; ++b) mn = fmaxf(mn, mb[b]), mon = fmaxf(mon, mb[b] + sc[b].y);
      // the sum's scale follows m exactly, the output's only in steps
      if (mn > m) l *= exp2f(m - mn), m = mn;
      const bool jump = mon > mo + kLazy;
      if (__any_sync(0xffffffffu, jump)) {
        const float f = mon > mo ? exp2f(mo - mon) : 1.f;
        mo = fmaxf(mo, mon);
        if (i > 0) {
          if (!(ok = wait_all(OD + t, (i - 1) & 1))) break;
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
    if (ok && nblk > 0 && (ok = wait_all(OD + t, (nblk - 1) & 1))) tc_fence_after();
    if (!ok) ctl->abort = 1;
    done_ok = ok;
  }

  // ---- output
  const bool alone = splits == 1;
  float* part = reinterpret_cast<float*>(a.ws + (((size_t)tiles * a.c.N * Hk * sizeof(unsigned) + 255) & ~(size_t)255));
  const int r = tid;  // row of the CTA (the first 256 threads)
  const int tt = (r0 + r) / G, head = hk * G + (r0 + r) % G;
  const bool in_call = tid < kRows && r0 + r < a.T * G;
  bf16* y = static_cast<bf16*>(a.y) + n * a.sy.n + head * a.sy.h + tt * a.sy.t;
  const bf16* add = a.add ? static_cast<const bf16*>(a.add) + n * a.sadd.n + head * a.sadd.h + tt * a.sadd.t : nullptr;
  // The meta tokens join a row's statistics; their logits stay for the values' weights.
  float zm[kMaxM];
  auto with_meta = [&](float& m_, float& l_) {
    const bf16* qp = static_cast<const bf16*>(a.q) + n * a.sq.n + head * a.sq.h + tt * a.sq.t;
    float top = m_;
#pragma unroll
    for (int j = 0; j < kMaxM; ++j) {
      zm[j] = -INFINITY;
      if (j < a.M) {
        const bf16* k = static_cast<const bf16*>(a.mk) + ((size_t)head * a.M + j) * D;
        float z = 0.f;
#pragma unroll 1
        for (int d = 0; d < D; d += 4) {
          const float4 x = ld4(qp + d), w = ld4(k + d);
          z += x.x * w.x + x.y * w.y + x.z * w.z + x.w * w.w;
        }
        zm[j] = z * a.scale * kLog2e;
        top = fmaxf(top, zm[j]);
      }
    }
    l_ = m_ == -INFINITY ? 0.f : l_ * exp2f(m_ - top);
#pragma unroll
    for (int j = 0; j < kMaxM; ++j)
      if (j < a.M) l_ += exp2f(zm[j] - top);
    m_ = top;
  };
  // Four channels of a row: o in units of 2^mo_, to be normalised by (m_, l_).
  auto finish = [&](float4 o, int d, float m_, float mo_, float l_) {
    const float f = l_ > 0.f && mo_ != -INFINITY ? a.alpha / l_ * exp2f(mo_ - m_) : 0.f;
    float4 v = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    if (f == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);  // o may hold nothing
    if (a.M > 0) {
      const float fm = l_ > 0.f ? a.alpha / l_ : 0.f;
#pragma unroll
      for (int j = 0; j < kMaxM; ++j)
        if (j < a.M) {
          const float w = exp2f(zm[j] - m_) * fm;
          const float4 x = ld4(static_cast<const bf16*>(a.mv) + ((size_t)head * a.M + j) * D + d);
          v.x = fmaf(w, x.x, v.x), v.y = fmaf(w, x.y, v.y), v.z = fmaf(w, x.z, v.z), v.w = fmaf(w, x.w, v.w);
        }
    }
    if (add) {
      const float4 x = ld4(add + d);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    return v;
  };
  const bool live = tid < kRows && r < rows && done_ok;
  if (warp < 8 && __all_sync(0xffffffffu, !*(volatile int*)&ctl->abort)) {
    const int t = warp >> 2;
    const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 + t * D;
    float m_ = m, l_ = l;
    if (alone && a.M > 0 && live) with_meta(m_, l_);
    float* mine = part + (size_t)blockIdx.x * kRows * (D + 4);
    if (!alone) *reinterpret_cast<float4*>(mine + (size_t)kRows * D + 4 * r) = make_float4(m, mo, l, 0.f);
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      uint32_t u[16];
      __syncwarp();
      if (nblk > 0) {
        tmem_ld16(to + c, u);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] = 0;
      }
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        float4 o = make_float4(__uint_as_float(u[e]), __uint_as_float(u[e + 1]), __uint_as_float(u[e + 2]),
                               __uint_as_float(u[e + 3]));
        if (!alone) *reinterpret_cast<float4*>(mine + (size_t)r * D + c + e) = o;
        else if (live) st4(y + c + e, finish(o, c + e, m_, mo, l_));
        else if (in_call) st4(y + c + e, make_float4(0.f, 0.f, 0.f, 0.f));
      }
    }
  }
  tc_fence_before();
  cta_sync();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (*(volatile int*)&ctl->abort) {
    if (tid == 0) raise_status(a.status, kDevTimeout);
  } else if (!alone) {
    __threadfence();
    __syncthreads();
    unsigned* counter = reinterpret_cast<unsigned*>(a.ws) + unit;
    if (tid == 0) s_last = atomicAdd(counter, 1u) == (unsigned)(splits - 1);
    __syncthreads();
    if (s_last && tid < kRows) {
      __threadfence();
      const float* p0 = part + (size_t)unit * splits * kRows * (D + 4);
      const size_t step = (size_t)kRows * (D + 4);
      float m_ = -INFINITY, mo_ = -INFINITY, l_ = 0.f;
      for (int s = 0; s < splits; ++s) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(p0 + s * step + (size_t)kRows * D + 4 * r));
        m_ = fmaxf(m_, x.x), mo_ = fmaxf(mo_, x.y);
      }
      for (int s = 0; s < splits; ++s) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(p0 + s * step + (size_t)kRows * D + 4 * r));
        if (x.x != -INFINITY) l_ += x.z * exp2f(x.x - m_);
      }
      if (r < rows && a.M > 0) with_meta(m_, l_);
      if (in_call)
#pragma unroll 1
        for (int d = 0; d < D; d += 4) {
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r < rows) {
            for (int s = 0; s < splits; ++s) {
              const float mos = __ldcg(p0 + s * step + (size_t)kRows * D + 4 * r + 1);
              if (mos == -INFINITY) continue;
              const float w = exp2f(mos - mo_);
              const float4 x = __ldcg(reinterpret_cast<const float4*>(p0 + s * step + (size_t)r * D + d));
              o.x = fmaf(w, x.x, o.x), o.y = fmaf(w, x.y, o.y), o.z = fmaf(w, x.z, o.z), o.w = fmaf(w, x.w, o.w);
            }
            o = finish(o, d, m_, mo_, l_);
          }
          st4(y + d, o);
        }
      if (tid == 0) *counter = 0u;
    }
  }
  pdl_trigger();
}

// CTAs of one wave; pieces a CTA's range is cut into when there are fewer CTAs than that.
constexpr int kWave = 152;
int split_count(int ctas) { return std::max(1, std::min(64, kWave / ctas)); }

template <int D, int F>
cudaError_t launch(const CacheAttn& a, cudaStream_t s, int* launches) {
  const int tiles = (a.H / a.c.Hk * a.T + kRows - 1) / kRows;
  const int64_t ctas = (int64_t)tiles * a.c.N * a.c.Hk;
  const int splits = ctas < kWave ? split_count((int)ctas) : 1;
  if (ctas * splits > 0x7fffffffll) return cudaErrorInvalidValue;
  constexpr int smem = Smem<D>::kBytes + 1024;
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D, F>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  trace_begin("cache_attn_prompt", s);
  e = launch_pdl(prompt_kernel<D, F>, dim3((unsigned)(ctas * splits)), dim3(kThreads), smem, s, a, tiles, splits);
  trace_end(s);
  ++*launches;
  return e;
}

}  // namespace

bool cache_attn_tc_used(int H, int Hk, int T, lizard_dtype dt) { return dt == LIZARD_BF16 && H / Hk * T > 128; }

size_t cache_attn_tc_workspace(int N, int Hk, int H, int T, int d) {
  const int tiles = (H / Hk * T + kRows - 1) / kRows;
  const int64_t ctas = (int64_t)tiles * N * Hk;
  const int splits = ctas < kWave ? split_count((int)ctas) : 1;
  const size_t counters = align_up((size_t)ctas * sizeof(unsigned), 256);
  return splits > 1 ? counters + (size_t)ctas * splits * kRows * (d + 4) * sizeof(float) : counters;
}

cudaError_t launch_cache_attn_tc(const CacheAttn& a, cudaStream_t s, int* launches) {
  if (a.c.d == 64)
    return a.c.fmt == LIZARD_KV_E4M3 ? launch<64, 0>(a, s, launches) : launch<64, 1>(a, s, launches);
  return a.c.fmt == LIZARD_KV_E4M3 ? launch<128, 0>(a, s, launches) : launch<128, 1>(a, s, launches);
}

}  // namespace lz
