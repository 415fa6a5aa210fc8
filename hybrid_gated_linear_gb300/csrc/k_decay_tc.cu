// k_decay_tc.cu -- one pass of the linear attention with a decay per head on the tensor cores (bf16),
// the state pass over segments of a long axis, and the products within a chunk that the gradient of
// log_decay needs.
//
// Chunks of 128 tokens, one after the other in the pass's direction; H the state that enters one:
//   S = A B^T,  P = S o D,  out = P C + from o (A H),  H' = all H + B^T (to o C)
// D the decays between the chunk's tokens, `from` and `to` those between a token and the chunk's edges.
// Every decay is a product of exponentials of sums of few log decays of one sign: for tokens of
// different 16-token blocks D = row (edge of its block to the one) G (blocks between) col, within
// a block the exponential of the running sum.  No difference of sums is formed, so minus infinity
// (a document's start) and very strong decays need no case of their own, and an element of P costs two
// multiplications instead of an exponential.
//
// A CTA takes 64 of C's channels of one head over the chunks of one segment; H stays in registers in
// fp32.  Twenty warps:
//   0      copies the tiles of A, B [128][da] and C [128][64] in by TMA, two stages ahead
//   1      issues the MMAs: S, B^T C~, A H, P C
//   2      the decays of the next chunk
//   4-11   C~ = to o C in two or three bf16 parts (16 or 24 bits: the state is a sum over the whole
//          sequence, so its operands are not rounded), then P, rounded once to bf16, into TMEM
//   12-19  the state: H = all H + (B^T C~); its bf16 parts for the next chunk's A H (one part, as P is
//          rounded too, or three where the product with H itself is a result); then the rows of out
// TMEM: S twice 2 x 128 columns, P 64, B^T C~ 64, P C 64, A H 64.
#include "lizard_dev.cuh"
#include "lizard_internal.h"
#include "tc_pipe.cuh"

namespace lz {
namespace {

using namespace tc;

constexpr int kC = kDecayTile;  // tokens of a chunk
constexpr int kN = 64;           // channels of c of a CTA
constexpr int kThreads = 640;
constexpr int kScoreWarps = 8, kStateWarps = 8;
constexpr int kTileC = kC * kN * 2;
constexpr int kColS = 0, kColP = 256, kColKV = 320, kColY = 384, kColYs = 448;

enum {
  FA = 0, FB = 2, FC = 4, EA = 6, EB = 8, EC = 10,  // tiles full and empty, by stage
  SR = 12,                                          // scores ready, by buffer
  CT = 14, KVR, KVF, HR, HF, PR, YR, YF, FACF, FACE, FIX, DONE, NB
};

struct alignas(16) Factors {
  float x[kC];    // log2 of the decays
  float row[kC], col[kC];
  float from[kC], to[kC];
  float g[64];    // [block of the output row][block of the source], the blocks between
  float all;
};

struct Head {  // in front of the tiles
  Ctl<NB> ctl;
  Factors f;
};
constexpr int kHead = 3072;
static_assert(sizeof(Head) <= kHead, "barriers and factors");

template <int DA, int NPH>
struct Smem {
  static constexpr int kTile = kC * DA * 2;
  static constexpr int NA = 2, NBt = DA == 128 && NPH == 3 ? 1 : 2, NCt = 2;
  static constexpr int A = 0, B = A + NA * kTile, Ct = B + NBt * kTile, CP = Ct + NCt * kTileC;
  static constexpr int kPartH = DA * kN * 2;
  static constexpr int H = CP + 3 * kTileC;
  static constexpr int kBytes = kHead + H + NPH * kPartH;
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

struct Maps {
  CUtensorMap a, b, c;
};

struct TcParams {
  DecayPass p;
  int an, ah, bn, bh, cn, ch;  // 0 where a tensor repeats over sequences or heads, else 1
  int segs, cps;               // segments of the axis, chunks of each
  int parts;                   // bf16 parts of C~
  bool states_only;            // first pass: the segments' states from zero
  float *seg_h, *seg_d;        // [segs][units][slices][da][64], [segs][units][slices]
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// D(tmem) (+)= A(tmem) * B(smem)^T ; issued by one thread.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  const uint32_t acc = accumulate ? 1u : 0u;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
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

__device__ __forceinline__ float f32(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Two values as sums of bf16 parts: the nearest, the nearest to what is left, and again.
__device__ __forceinline__ void split(float a, float b, uint32_t (&o)[3]) {
  o[0] = pack_bf16x2(a, b);
  a -= lo_f(o[0]), b -= hi_f(o[0]);
  o[1] = pack_bf16x2(a, b);
  a -= lo_f(o[1]), b -= hi_f(o[1]);
  o[2] = pack_bf16x2(a, b);
}

// One warp: the factors of a chunk from its log decays (log2, minus infinity where a document starts),
// four tokens a lane, four lanes a block.
__device__ __forceinline__ void make_factors(const float (&x)[4], float (&pre)[4], float (&suf)[4], float (&in)[4],
                                             float (&out)[4], float (&g)[2], float& all) {
  const int lane = threadIdx.x & 31;
  pre[0] = x[0], pre[1] = pre[0] + x[1], pre[2] = pre[1] + x[2], pre[3] = pre[2] + x[3];
  suf[3] = 0.f, suf[2] = x[3], suf[1] = suf[2] + x[2], suf[0] = suf[1] + x[1];
  float up = pre[3], down = pre[3];
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const float u = __shfl_up_sync(0xffffffffu, up, o, 4), d = __shfl_down_sync(0xffffffffu, down, o, 4);
    if ((lane & 3) >= o) up += u;
    if ((lane & 3) + o < 4) down += d;
  }
  float before = __shfl_up_sync(0xffffffffu, up, 1, 4), behind = __shfl_down_sync(0xffffffffu, down, 1, 4);
  if ((lane & 3) == 0) before = 0.f;
  if ((lane & 3) == 3) behind = 0.f;
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = __shfl_sync(0xffffffffu, up, 4 * j + 3);
  float head = 0.f, tail = 0.f, sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j < (lane >> 2)) head += t[j];
    if (j > (lane >> 2)) tail += t[j];
    sum += t[j];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float p = pre[k] + before, s = suf[k] + behind;
    pre[k] = exp2f(p), suf[k] = exp2f(s);
    in[k] = exp2f(p + head), out[k] = exp2f(s + tail);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = (lane >> 3) + 4 * e, j = lane & 7;
    float between = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k > min(i, j) && k < max(i, j)) between += t[k];
    g[e] = exp2f(between);
  }
  all = exp2f(sum);
}

// Four of a chunk's log decays in log2 (a lane's own); past the sequence's end 0.
__device__ __forceinline__ void load_decays(const float* lg, int64_t st, int t0, int count, float (&x)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = t0 + 4 * lane + k;
    const float g = t < count ? lg[t * st] : 0.f;
    x[k] = g < kDecayNone ? -INFINITY : g * 1.4426950408889634f;
  }
}

__device__ __forceinline__ void store_factors(Factors& f, bool rev, const float (&x)[4], const float (&pre)[4], const float (&suf)[4],
                                              const float (&in)[4], const float (&out)[4], const float (&g)[2], float all) {
  const int lane = threadIdx.x & 31;
  auto put = [&](float* d, const float (&v)[4]) {
    *reinterpret_cast<float4*>(d + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
  };
  put(f.x, x);
  put(rev ? f.col : f.row, pre);
  put(rev ? f.row : f.col, suf);
  put(rev ? f.to : f.from, in);
  put(rev ? f.from : f.to, out);
  f.g[lane] = g[0], f.g[lane + 32] = g[1];
  if (lane == 0) f.all = all;
}

// The decays within a 16-token block between token `o` of it and each token s, s <= o (s >= o with
// rev) and 0 elsewhere; x: the block's log2 decays.
__device__ __forceinline__ void block_decays(const float* x, int o, bool rev, float (&d)[16]) {
  float v[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 q = *reinterpret_cast<const float4*>(x + 4 * j);
    v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
  }
  float sum = 0.f;
  if (rev) {
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      sum = s <= o ? 0.f : sum + v[s];
      d[s] = s < o ? 0.f : ex2_approx(sum);
    }
  } else {
#pragma unroll
    for (int s = 15; s >= 0; --s) {
      sum = s >= o ? 0.f : sum + v[s < 15 ? s + 1 : 15];
      d[s] = s > o ? 0.f : ex2_approx(sum);
    }
  }
}

// 16 values to a row of out, as bf16 or fp32.
__device__ __forceinline__ void put_row(void* out, int64_t at, bool wide, const float (&v)[16]) {
  if (wide) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
    uint4* d = reinterpret_cast<uint4*>(static_cast<bf16*>(out) + at);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      d[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                        pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
  }
}

template <int DA, int NPH>
__global__ void __launch_bounds__(kThreads, 1)
    decay_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ TcParams q) {
  using Sm = Smem<DA, NPH>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const DecayPass& p = q.p;
  Head& hd = *reinterpret_cast<Head*>(smem_raw);
  Ctl<NB>* ctl = &hd.ctl;
  unsigned char* sm = smem_raw + kHead;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // tiles of the 128-byte swizzle start on 1024 bytes: so does the dynamic part where there is no
  // static one; anything else would be caught here, not computed with
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (tid == 0) raise_status(p.status, kDevCheck);
    return;
  }
  const int slices = p.dc / kN, units = p.B * p.H;
  const int slice = blockIdx.x % slices, unit = blockIdx.x / slices % units, seg = blockIdx.x / slices / units;
  const int n = unit / p.H, h = unit - n * p.H, c0 = slice * kN;

  if (warp == 1) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = FA; i < CT; ++i) mbar_init(&ctl->bar[i], 1);
    mbar_init(&ctl->bar[CT], kScoreWarps), mbar_init(&ctl->bar[PR], kScoreWarps), mbar_init(&ctl->bar[FIX], kScoreWarps);
    mbar_init(&ctl->bar[HR], kStateWarps), mbar_init(&ctl->bar[KVF], kStateWarps), mbar_init(&ctl->bar[YF], kStateWarps);
    mbar_init(&ctl->bar[KVR], 1), mbar_init(&ctl->bar[HF], 1), mbar_init(&ctl->bar[YR], 1), mbar_init(&ctl->bar[DONE], 1);
    mbar_init(&ctl->bar[FACF], 1), mbar_init(&ctl->bar[FACE], kScoreWarps + kStateWarps);
    ctl->abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  pdl_wait();

  int count = p.L;
  if (p.count) {
    count = p.count[n];
    if (count < 0 || count > p.L) {
      if (tid == 0) raise_status(p.status, kDevCheck);
      count = 0;
    }
  }
  // this segment's chunks, in the pass's order from `first` on
  const int chunks = (count + kC - 1) / kC;
  const int done = min(seg * q.cps, chunks), num = min(q.cps, chunks - done);
  const int first = p.rev ? chunks - 1 - done : done, dir = p.rev ? -1 : 1;
  auto token = [&](int it) { return (first + dir * it) * kC; };
  // the one chunk whose last rows lie behind the sequence but inside the tensor: they are zeroed
  // before any product, as they may hold anything
  auto ragged = [&](int it) { return token(it) + kC > count && count < p.L; };

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      uint32_t armed_a[2] = {0, 0}, armed_b[2] = {0, 0}, armed_c[2] = {0, 0};
      const int na = q.an * n, nb = q.bn * n, nc = q.cn * n, ha = q.ah * (h / p.ga), hb = q.bh * (h / p.gb),
                hc = q.ch * (h / p.gc);
      for (int it = 0; it < num && ok; ++it) {
        const int t0 = token(it);
        const int sc = it % Sm::NCt, sb = it % Sm::NBt, sa = it % Sm::NA;
        if (it >= Sm::NCt && !(ok = wait_bar(ctl, EC + sc, (it / Sm::NCt - 1) & 1))) break;
        mbar_arrive_expect_tx(&ctl->bar[FC + sc], kTileC);
        tma_load_4d(sm + Sm::Ct + sc * kTileC, &maps.c, c0, t0, hc, nc, &ctl->bar[FC + sc]);
        armed_c[0] += sc == 0, armed_c[1] += sc == 1;
        if (it >= Sm::NBt && !(ok = wait_bar(ctl, EB + sb, (it / Sm::NBt - 1) & 1))) break;
        mbar_arrive_expect_tx(&ctl->bar[FB + sb], Sm::kTile);
#pragma unroll
        for (int k = 0; k < DA / 64; ++k)
          tma_load_4d(sm + Sm::B + sb * Sm::kTile + k * (kC * 128), &maps.b, 64 * k, t0, hb, nb, &ctl->bar[FB + sb]);
        armed_b[0] += sb == 0, armed_b[1] += sb == 1;
        if (q.states_only) continue;
        if (it >= Sm::NA && !(ok = wait_bar(ctl, EA + sa, (it / Sm::NA - 1) & 1))) break;
        mbar_arrive_expect_tx(&ctl->bar[FA + sa], Sm::kTile);
#pragma unroll
        for (int k = 0; k < DA / 64; ++k)
          tma_load_4d(sm + Sm::A + sa * Sm::kTile + k * (kC * 128), &maps.a, 64 * k, t0, ha, na, &ctl->bar[FA + sa]);
        armed_a[0] += sa == 0, armed_a[1] += sa == 1;
      }
      if (!ok) ctl->abort = 1;
      const uint64_t t0 = globaltimer_ns();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        drain_bar(ctl, FA + k, armed_a[k], t0);
        drain_bar(ctl, FB + k, armed_b[k], t0);
        drain_bar(ctl, FC + k, armed_c[k], t0);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t sb = smem_u32(sm);
      const uint32_t id_s = idesc_bf16(kC, kC, false, false), id_kv = idesc_bf16(128, kN, true, true),
                     id_h = idesc_bf16(kC, kN, false, true);
      bool ok = true;
      auto scores = [&](int it) {  // S = A B^T
        if (!wait_bar(ctl, FA + it % Sm::NA, (it / Sm::NA) & 1) || !wait_bar(ctl, FB + it % Sm::NBt, (it / Sm::NBt) & 1))
          return false;
        if (ragged(it) && !wait_bar(ctl, FIX, 0)) return false;
        tc_fence_after();
        const uint32_t ta = sb + Sm::A + it % Sm::NA * Sm::kTile, tb = sb + Sm::B + it % Sm::NBt * Sm::kTile;
#pragma unroll
        for (int j = 0; j < DA / 16; ++j)
          mma_bf16(tmem + kColS + (it & 1) * 128, desc_k(ta, kC, j), desc_k(tb, kC, j), id_s, j > 0);
        mma_commit(&ctl->bar[SR + (it & 1)]);
        return true;
      };
      if (num > 0 && !q.states_only) ok = scores(0);
      for (int it = 0; it < num && ok; ++it) {
        const uint32_t tb = sb + Sm::B + it % Sm::NBt * Sm::kTile, tc_ = sb + Sm::Ct + it % Sm::NCt * kTileC;
        // B^T C~ (the B tile is there: its scores are, or it is waited for)
        if (!(ok = wait_bar(ctl, CT, it & 1))) break;
        if (q.states_only && !(ok = wait_bar(ctl, FB + it % Sm::NBt, (it / Sm::NBt) & 1))) break;
        if (it > 0 && !(ok = wait_bar(ctl, KVF, (it - 1) & 1))) break;
        tc_fence_after();
        // (the smallest parts first, while the sum and what its additions cut off are small)
        for (int k = q.parts - 1; k >= 0; --k) {
          const uint32_t tp = sb + Sm::CP + k * kTileC;
#pragma unroll
          for (int j = 0; j < kC / 16; ++j)
            mma_bf16(tmem + kColKV, desc_mn(tb, kC, j), desc_mn(tp, kC, j), id_kv, k < q.parts - 1 || j > 0);
        }
        mma_commit(&ctl->bar[KVR]);
        mma_commit(&ctl->bar[EB + it % Sm::NBt]);
        if (q.states_only) {
          mma_commit(&ctl->bar[EC + it % Sm::NCt]);
          continue;
        }
        // the next chunk's scores go first where their B tile can be there already
        if (Sm::NBt > 1 && it + 1 < num && !(ok = scores(it + 1))) break;
        // A H
        if (!(ok = wait_bar(ctl, HR, it & 1))) break;
        if (it > 0 && !(ok = wait_bar(ctl, YF, (it - 1) & 1))) break;
        tc_fence_after();
        const uint32_t ta = sb + Sm::A + it % Sm::NA * Sm::kTile;
#pragma unroll
        for (int k = NPH - 1; k >= 0; --k)
#pragma unroll
          for (int j = 0; j < DA / 16; ++j)
            mma_bf16(tmem + kColYs, desc_k(ta, kC, j), desc_mn(sb + Sm::H + k * Sm::kPartH, DA, j), id_h, k < NPH - 1 || j > 0);
        mma_commit(&ctl->bar[HF]);
        mma_commit(&ctl->bar[EA + it % Sm::NA]);
        // P C
        if (!(ok = wait_bar(ctl, PR, it & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
          mma_bf16_ts(tmem + kColY, tmem + kColP + 8 * j, desc_mn(tc_, kC, j), id_h, j > 0);
        mma_commit(&ctl->bar[YR]);
        mma_commit(&ctl->bar[EC + it % Sm::NCt]);
        if (Sm::NBt == 1 && it + 1 < num) ok = scores(it + 1);
      }
      if (!ok) ctl->abort = 1;
      mma_commit(&ctl->bar[DONE]);
      drain_bar(ctl, DONE, 1, globaltimer_ns());
    }
  } else if (warp == 2) {
    const float* lg = p.lg + n * p.sg.n + h * p.sg.h;
    float x[4], nx[4] = {};
    if (num > 0) load_decays(lg, p.sg.t, token(0), count, x);
    for (int it = 0; it < num; ++it) {
      float pre[4], suf[4], in[4], out[4], g[2], all;
      if (it + 1 < num) load_decays(lg, p.sg.t, token(it + 1), count, nx);
      make_factors(x, pre, suf, in, out, g, all);
      if (it > 0 && !wait_bar(ctl, FACE, (it - 1) & 1)) break;
      store_factors(hd.f, p.rev, x, pre, suf, in, out, g, all);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[FACF]);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = nx[k];
    }
  } else if (warp >= 4 && warp < 12) {
    const int half = (warp - 4) >> 2, qw = warp & 3, wt = tid - 128;  // thread of the group
    const int o = 32 * qw + lane, I = o >> 4;
    const uint32_t tl = (uint32_t)(qw * 32) << 16;
    const Factors& f = hd.f;
    if (!q.states_only) {  // the part of P that is always 0
      const uint32_t z[16] = {};
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if ((g & 1) == half && (p.rev ? g < qw : g > qw)) tmem_st16(tmem + tl + kColP + 16 * g, z);
      tmem_st_wait();
    }
    bool ok = true;
    for (int it = 0; it < num && ok; ++it) {
      const int valid = min(kC, count - token(it));
      unsigned char* tc_ = sm + Sm::Ct + it % Sm::NCt * kTileC;
      if (!(ok = wait_bar(ctl, FC + it % Sm::NCt, (it / Sm::NCt) & 1))) break;
      if (ragged(it)) {
        if (!(ok = wait_bar(ctl, FB + it % Sm::NBt, (it / Sm::NBt) & 1))) break;
        unsigned char* tb = sm + Sm::B + it % Sm::NBt * Sm::kTile;
        const uint4 z = make_uint4(0, 0, 0, 0);
        // (each thread the same places of C that it reads below)
        for (int at = wt * 16; at < kTileC; at += 32 * kScoreWarps * 16) {
          if (at < valid * 128) continue;
          *reinterpret_cast<uint4*>(tc_ + at) = z;
#pragma unroll
          for (int k = 0; k < DA / 64; ++k) *reinterpret_cast<uint4*>(tb + k * (kC * 128) + at) = z;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->bar[FIX]);
      }
      if (!(ok = wait_bar(ctl, FACF, it & 1))) break;
      // C~ (its tiles are free once the chunk before has been multiplied)
      if (it > 0 && !(ok = wait_bar(ctl, KVR, (it - 1) & 1))) break;
#pragma unroll
      for (int e = 0; e < kTileC / 16 / (32 * kScoreWarps); ++e) {
        const int at = (wt + 32 * kScoreWarps * e) * 16;  // byte of the tile: the swizzle stays as it is
        const float w = f.to[at >> 7] * p.scale_in;
        const uint4 v = *reinterpret_cast<const uint4*>(tc_ + at);
        uint32_t o0[3], o1[3], o2[3], o3[3];
        split(w * lo_f(v.x), w * hi_f(v.x), o0);
        split(w * lo_f(v.y), w * hi_f(v.y), o1);
        split(w * lo_f(v.z), w * hi_f(v.z), o2);
        split(w * lo_f(v.w), w * hi_f(v.w), o3);
        unsigned char* d = sm + Sm::CP + at;
        *reinterpret_cast<uint4*>(d) = make_uint4(o0[0], o1[0], o2[0], o3[0]);
        *reinterpret_cast<uint4*>(d + kTileC) = make_uint4(o0[1], o1[1], o2[1], o3[1]);
        if (q.parts > 2) *reinterpret_cast<uint4*>(d + 2 * kTileC) = make_uint4(o0[2], o1[2], o2[2], o3[2]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[CT]);
      if (q.states_only) {
        if (lane == 0) mbar_arrive(&ctl->bar[FACE]);
        continue;
      }
      // P
      if (!(ok = wait_bar(ctl, SR + (it & 1), (it >> 1) & 1))) break;
      if (it > 0 && !(ok = wait_bar(ctl, YR, (it - 1) & 1))) break;
      tc_fence_after();
      const float rf = f.row[o] * p.scale_in;
#pragma unroll 1
      for (int g = half; g < 4; g += 2) {
        if (p.rev ? g < qw : g > qw) continue;
        uint32_t s[32], w[16];
        tmem_ld32(tmem + tl + kColS + (it & 1) * 128 + 32 * g, s);
        if (g != qw) {
          tmem_ld_wait();
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float r = rf * f.g[I * 8 + 2 * g + b];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 c = *reinterpret_cast<const float4*>(&f.col[32 * g + 16 * b + 4 * j]);
              w[8 * b + 2 * j] = pack_bf16x2(f32(s[16 * b + 4 * j]) * (r * c.x), f32(s[16 * b + 4 * j + 1]) * (r * c.y));
              w[8 * b + 2 * j + 1] = pack_bf16x2(f32(s[16 * b + 4 * j + 2]) * (r * c.z), f32(s[16 * b + 4 * j + 3]) * (r * c.w));
            }
          }
        } else {
          float d[16];
          block_decays(f.x + 16 * I, lane & 15, p.rev, d);
          tmem_ld_wait();
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const bool own = (lane >> 4) == b;
            // the other block of the pair: seen by the later tokens (the earlier ones with rev)
            const float r = (p.rev ? b == 1 : b == 0) ? rf : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 c = *reinterpret_cast<const float2*>(&f.col[32 * g + 16 * b + 2 * j]);
              const float d0 = own ? d[2 * j] * p.scale_in : r * c.x, d1 = own ? d[2 * j + 1] * p.scale_in : r * c.y;
              w[8 * b + j] = pack_bf16x2(f32(s[16 * b + 2 * j]) * d0, f32(s[16 * b + 2 * j + 1]) * d1);
            }
          }
        }
        tmem_st16(tmem + tl + kColP + 16 * g, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[PR]), mbar_arrive(&ctl->bar[FACE]);
    }
    if (!ok) ctl->abort = 1;
  } else if (warp >= 12) {
    const int half = (warp - 12) >> 2, qw = warp & 3;
    const int i = 32 * qw + lane;  // row of the state, row of the output
    const bool mine = i < DA;
    const uint32_t tl = tmem + ((uint32_t)(qw * 32) << 16) + 32 * half;
    const Factors& f = hd.f;
    float x[32];
    auto at = [&](int j) {  // column j of this thread in a state of the caller's
      const int c = c0 + 32 * half + j;
      return (int64_t)unit * DA * p.dc + (p.state_t ? (int64_t)c * DA + i : (int64_t)i * p.dc + c);
    };
    float* seg_h = q.seg_h + ((((int64_t)seg * units + unit) * slices + slice) * DA + i) * kN + 32 * half;
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = 0.f;
    if (mine && !q.states_only) {
      if (q.segs > 1) {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = seg_h[j];
      } else if (p.init) {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = p.init[at(j)];
      }
    }
    auto put_state = [&]() {  // the parts of H for A H: rows of 64 channels, swizzled
      if (mine) {
        unsigned char* d = sm + Sm::H + i * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t o[4][3];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (NPH == 1)
              o[k][0] = pack_bf16x2(x[8 * j + 2 * k], x[8 * j + 2 * k + 1]);
            else
              split(x[8 * j + 2 * k], x[8 * j + 2 * k + 1], o[k]);
          }
          const int c = ((4 * half + j) ^ (i & 7)) * 16;
#pragma unroll
          for (int k = 0; k < NPH; ++k)
            *reinterpret_cast<uint4*>(d + k * Sm::kPartH + c) = make_uint4(o[0][k], o[1][k], o[2][k], o[3][k]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[HR]);
    };
    const int64_t so = n * p.so.n + h * p.so.h + c0 + 32 * half;
    const bf16* px = p.x ? static_cast<const bf16*>(p.x) + n * p.sx.n + h / p.gx * p.sx.h + c0 + 32 * half : nullptr;
    float* dot = p.x ? p.dot_out + ((int64_t)(2 * slice + half) * units + unit) * p.L : nullptr;
    bool ok = true;
    float product = 1.f;
    if (num > 0 && !q.states_only) put_state();
    for (int it = 0; it < num && ok; ++it) {
      if (!(ok = wait_bar(ctl, FACF, it & 1))) break;
      const float from = f.from[i], all = f.all;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[FACE]);
      product *= all;
      // H = all H + B^T C~
      if (!(ok = wait_bar(ctl, KVR, it & 1))) break;
      tc_fence_after();
      {
        uint32_t kv[32];
        tmem_ld32(tl + kColKV, kv);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->bar[KVF]);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = fmaf(all, x[j], f32(kv[j]));
      }
      if (q.states_only) continue;
      if (it + 1 < num) {
        if (!(ok = wait_bar(ctl, HF, it & 1))) break;
        put_state();
      }
      // out = P C + from o (A H)
      const int t = token(it) + i;
      const bool live = t < count;
      if (!(ok = wait_bar(ctl, YR, it & 1))) break;
      tc_fence_after();
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t y[16], ys[16];
        tmem_ld16(tl + kColY + 16 * e, y);
        tmem_ld16(tl + kColYs + 16 * e, ys);
        tmem_ld_wait();
        if (e == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->bar[YF]);
        }
        float v[16];
        if (px && live) {
          const uint4* xr = reinterpret_cast<const uint4*>(px + t * p.sx.t + 16 * e);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 u = xr[k];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              d = fmaf(lo_f(w[r]), f32(ys[8 * k + 2 * r]), d);
              d = fmaf(hi_f(w[r]), f32(ys[8 * k + 2 * r + 1]), d);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = live ? p.scale_out * fmaf(from, f32(ys[j]), f32(y[j])) : 0.f;
        if (t < p.L) put_row(p.out, so + t * p.so.t + 16 * e, p.out_f32, v);
      }
      if (px && live) dot[t] = p.scale_out * from * d;
    }
    if (!ok) ctl->abort = 1;
    if (ok && q.states_only) {
      if (mine) {
#pragma unroll
        for (int j = 0; j < 32; ++j) seg_h[j] = x[j];
      }
      if (i == 0 && half == 0) q.seg_d[((int64_t)seg * units + unit) * slices + slice] = product;
    } else if (ok) {
      if (mine && p.fin && seg == q.segs - 1) {
#pragma unroll
        for (int j = 0; j < 32; ++j) p.fin[at(j)] = x[j];
      }
      // the rows of whole chunks behind the sequence
      const int all_chunks = (p.L + kC - 1) / kC;
      const int za = max(seg * q.cps, chunks), zb = min((seg + 1) * q.cps, all_chunks);
      const float z[16] = {};
      for (int c = za; c < zb; ++c) {
        const int t = c * kC + i;
        if (t < p.L) {
          put_row(p.out, so + t * p.so.t, p.out_f32, z);
          put_row(p.out, so + t * p.so.t + 16, p.out_f32, z);
        }
      }
    }
  }
  tc_fence_before();
  cta_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && ctl->abort) raise_status(p.status, kDevTimeout);
}

// The segments' starting states in place of their own states: cur = init; for each segment its slot
// becomes cur, and cur = decay cur + the segment's state.
__global__ void __launch_bounds__(256) decay_join_kernel(DecayPass p, int segs, float* seg_h, const float* seg_d) {
  pdl_wait();
  const int slices = p.dc / kN, units = p.B * p.H;
  const int64_t per = (int64_t)p.da * kN, total = (int64_t)units * slices * per;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= total) return;
  const int64_t us = e / per;
  const int unit = (int)(us / slices), slice = (int)(us - (int64_t)unit * slices);
  const int r = (int)(e - us * per), i = r / kN, c = slice * kN + r % kN;
  float cur = p.init ? p.init[(int64_t)unit * p.da * p.dc + (p.state_t ? (int64_t)c * p.da + i : (int64_t)i * p.dc + c)] : 0.f;
  for (int s = 0; s < segs; ++s) {
    float* slot = seg_h + s * total + e;
    const float own = s + 1 < segs ? *slot : 0.f, d = s + 1 < segs ? seg_d[(int64_t)s * units * slices + us] : 0.f;
    *slot = cur;
    cur = fmaf(d, cur, own);
  }
}

// ---------------------------------------------------------------------------------
// Within a chunk: row_i = sum_{s < i} W_is, col_s = sum_{i > s} W_is with W_is = scale (q_i . k_s) D (dy_i . v_s),
// from exact products of the bf16 rows in fp32 sums.  One CTA a chunk: both scores and their transposes by
// four MMAs; four warps sum the rows, four the columns, each thread its own.
// ---------------------------------------------------------------------------------
constexpr int kPairThreads = 384;
enum { GF = 0, GS, GT, GN };
struct PairMaps {
  CUtensorMap q, k, v, y;
};
struct PairParams {
  int B, H, L, G;  // G: query heads per key head
  int qn, qh, kn, kh, vn, vh, yn, yh;
  const float* lg;
  Strides sg;
  const int32_t* count;
  float scale;
  float *row, *col;  // [B,H,L]
  unsigned* status;
};
template <int DK, int DV>
struct PairSmem {
  static constexpr int kQ = kC * DK * 2, kV = kC * DV * 2;
  static constexpr int Q = 0, K = kQ, V = 2 * kQ, Y = V + kV, kBytes = kHead + Y + kV;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kPairThreads, 1)
    decay_pairs_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams p, int chunks) {
  using Sm = PairSmem<DK, DV>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Ctl<GN>* ctl = reinterpret_cast<Ctl<GN>*>(smem_raw);
  Factors& f = *reinterpret_cast<Factors*>(smem_raw + 64);
  static_assert(sizeof(Ctl<GN>) <= 64 && 64 + sizeof(Factors) <= kHead, "barriers and factors");
  unsigned char* sm = smem_raw + kHead;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (tid == 0) raise_status(p.status, kDevCheck);
    return;
  }
  const int unit = blockIdx.x / chunks, t0 = (blockIdx.x - unit * chunks) * kC;
  const int n = unit / p.H, h = unit - n * p.H;
  pdl_wait();
  int count = p.count ? p.count[n] : p.L;
  if (count < 0 || count > p.L) count = 0;  // flagged by the passes
  if (t0 >= count) return;
  if (warp == 1) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < GN; ++i) mbar_init(&ctl->bar[i], 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  if (warp == 0) {
    if (lane == 0) {
      uint64_t* bar = &ctl->bar[GF];
      mbar_arrive_expect_tx(bar, 2 * (Sm::kQ + Sm::kV));
      const int hk = h / p.G;
#pragma unroll
      for (int k = 0; k < DK / 64; ++k) {
        tma_load_4d(sm + Sm::Q + k * kC * 128, &maps.q, 64 * k, t0, p.qh * h, p.qn * n, bar);
        tma_load_4d(sm + Sm::K + k * kC * 128, &maps.k, 64 * k, t0, p.kh * hk, p.kn * n, bar);
      }
#pragma unroll
      for (int k = 0; k < DV / 64; ++k) {
        tma_load_4d(sm + Sm::V + k * kC * 128, &maps.v, 64 * k, t0, p.vh * hk, p.vn * n, bar);
        tma_load_4d(sm + Sm::Y + k * kC * 128, &maps.y, 64 * k, t0, p.yh * h, p.yn * n, bar);
      }
      drain_bar(ctl, GF, 1, globaltimer_ns());
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t sb = smem_u32(sm), id = idesc_bf16(kC, kC, false, false);
      bool ok = wait_bar(ctl, GF, 0);
      if (ok) {
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < DK / 16; ++j) mma_bf16(tmem, desc_k(sb + Sm::Q, kC, j), desc_k(sb + Sm::K, kC, j), id, j > 0);
#pragma unroll
        for (int j = 0; j < DV / 16; ++j) mma_bf16(tmem + 128, desc_k(sb + Sm::Y, kC, j), desc_k(sb + Sm::V, kC, j), id, j > 0);
        mma_commit(&ctl->bar[GS]);
#pragma unroll
        for (int j = 0; j < DK / 16; ++j)
          mma_bf16(tmem + 256, desc_k(sb + Sm::K, kC, j), desc_k(sb + Sm::Q, kC, j), id, j > 0);
#pragma unroll
        for (int j = 0; j < DV / 16; ++j)
          mma_bf16(tmem + 384, desc_k(sb + Sm::V, kC, j), desc_k(sb + Sm::Y, kC, j), id, j > 0);
      } else {
        ctl->abort = 1;
      }
      mma_commit(&ctl->bar[GT]);
      drain_bar(ctl, GT, 1, globaltimer_ns());
    }
  } else if (warp >= 4) {
    const bool rev = warp >= 8;  // the columns: token s receives from the later ones
    const int qw = warp & 3, o = 32 * qw + lane, I = o >> 4;
    if (warp == 4) {
      float x[4], pre[4], suf[4], in[4], out[4], g[2], all;
      load_decays(p.lg + n * p.sg.n + h * p.sg.h, p.sg.t, t0, count, x);
      make_factors(x, pre, suf, in, out, g, all);
      store_factors(f, false, x, pre, suf, in, out, g, all);
    }
    named_sync(1, 256);
    const float* rowf = rev ? f.col : f.row;
    const float* colf = rev ? f.row : f.col;
    const uint32_t tl = tmem + ((uint32_t)(qw * 32) << 16) + (rev ? 256 : 0);
    const bool ok = wait_bar(ctl, rev ? GT : GS, 0);
    if (ok) {
      tc_fence_after();
      const float rf = rowf[o];
      float sum = 0.f;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        if (rev ? g < qw : g > qw) continue;
        uint32_t s[32], y[32];
        tmem_ld32(tl + 32 * g, s);
        tmem_ld32(tl + 128 + 32 * g, y);
        float d[16];
        if (g == qw) block_decays(f.x + 16 * I, lane & 15, rev, d);
        tmem_ld_wait();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const bool own = g == qw && (lane >> 4) == b;
          const float r = g != qw ? rf * f.g[I * 8 + 2 * g + b] : (rev ? b == 1 : b == 0) ? rf : 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int e = 32 * g + 16 * b + j;
            const float w = own ? (e == o ? 0.f : d[j]) : r * colf[e];
            // (a decay of 0 hides the token, and rows behind the sequence may hold anything)
            const float v = f32(s[16 * b + j]) * f32(y[16 * b + j]);
            sum += w != 0.f && t0 + e < count ? w * v : 0.f;
          }
        }
      }
      const int t = t0 + o;
      if (t < count) (rev ? p.col : p.row)[(int64_t)unit * p.L + t] = p.scale * sum;
    } else {
      ctl->abort = 1;
    }
  }
  tc_fence_before();
  cta_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && ctl->abort) raise_status(p.status, kDevTimeout);
}

// A tensor of rows as the tensor map takes it: axes of one entry, or repeated ones, have extent 1.
bool rows_map(CUtensorMap* m, const void* base, int64_t B, int64_t H, int64_t L, int d, const Strides& s, int* kn, int* kh) {
  *kn = B > 1 && s.n > 0, *kh = H > 1 && s.h > 0;
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)L, *kh ? (uint64_t)H : 1, *kn ? (uint64_t)B : 1};
  const uint64_t st[3] = {L > 1 ? (uint64_t)s.t * 2 : 16 * 16, *kh ? (uint64_t)s.h * 2 : 16 * 16, *kn ? (uint64_t)s.n * 2 : 16 * 16};
  return make_tma_map_4d_bf16(m, base, dims, st, 64, kC);
}
bool strides_ok(int64_t B, int64_t H, int64_t L, int d, const Strides& s) {
  const int64_t most = 1ll << 38;  // elements: a stride of a map is below 2^40 bytes
  return (B <= 1 || s.n < most) && (H <= 1 || s.h < most) && (L <= 1 || (s.t >= d && s.t < most));
}

template <int DA, int NPH>
cudaError_t launch(const Maps& m, const TcParams& q, int blocks, cudaStream_t s) {
  using Sm = Smem<DA, NPH>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(decay_tc_kernel<DA, NPH>, Sm::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(decay_tc_kernel<DA, NPH>, dim3(blocks), dim3(kThreads), Sm::kBytes, s, m, q);
}

template <int DK, int DV>
cudaError_t launch_pairs(const PairMaps& m, const PairParams& p, cudaStream_t s) {
  using Sm = PairSmem<DK, DV>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(decay_pairs_kernel<DK, DV>, Sm::kBytes, done);
  if (e != cudaSuccess) return e;
  const int chunks = (p.L + kC - 1) / kC;
  const int64_t blocks = (int64_t)p.B * p.H * chunks;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_pdl(decay_pairs_kernel<DK, DV>, dim3((unsigned)blocks), dim3(kPairThreads), Sm::kBytes, s, m, p, chunks);
}

}  // namespace

bool decay_tc_rows_ok(int B, int H, int L, int d, const Strides& s) { return strides_ok(B, H, L, d, s); }

// Segments of the axis: CTAs run one to an SM (152), so that `ctas` of them take ceil(ctas S / 152) rounds of
// ceil(chunks / S) chunks, and before that, for S > 1, the states of all segments but the last, at
// about half the time a chunk, and a join.
int decay_segments(int ctas, int chunks) {
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= 32 && s <= chunks; ++s) {
    const int cps = (chunks + s - 1) / s;
    if (s > 1 && (chunks + cps - 1) / cps < s) continue;  // some would be empty
    double t = (double)(((int64_t)ctas * s + 151) / 152) * (cps + 2);
    if (s > 1) t += 0.5 * (double)(((int64_t)ctas * (s - 1) + 151) / 152) * (cps + 2) + 4;
    if (t < least) least = t, best = s;
  }
  return best;
}

size_t decay_tc_workspace(int B, int H, int L, int da, int dc) {
  const int64_t ctas = (int64_t)B * H * (dc / kN);
  const int segs = ctas > 152 * 32 ? 1 : decay_segments((int)ctas, (L + kC - 1) / kC);
  return segs > 1 ? (size_t)segs * ctas * ((size_t)da * kN + 1) * sizeof(float) : 0;
}

cudaError_t launch_decay_tc(const DecayPass& a, bool exact_state, float* ws, cudaStream_t s, int* launches) {
  Maps m;
  TcParams q{};
  q.p = a;
  if (!rows_map(&m.a, a.a, a.B, a.H / a.ga, a.L, a.da, a.sa, &q.an, &q.ah) ||
      !rows_map(&m.b, a.b, a.B, a.H / a.gb, a.L, a.da, a.sb, &q.bn, &q.bh) ||
      !rows_map(&m.c, a.c, a.B, a.H / a.gc, a.L, a.dc, a.sc, &q.cn, &q.ch))
    return cudaErrorInvalidValue;
  const int64_t ctas = (int64_t)a.B * a.H * (a.dc / kN);
  const int chunks = (a.L + kC - 1) / kC;
  q.segs = ctas > 152 * 32 ? 1 : decay_segments((int)ctas, chunks);
  q.cps = (chunks + q.segs - 1) / q.segs;
  q.parts = a.fin || a.x ? 3 : 2;
  if (ctas * q.segs > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaError_t e;
  if (q.segs > 1) {
    q.seg_h = ws, q.seg_d = ws + q.segs * ctas * a.da * kN;
    TcParams f = q;
    f.states_only = true;
    trace_begin("decay_states", s);
    e = a.da == 64 ? launch<64, 1>(m, f, (int)(ctas * (q.segs - 1)), s) : launch<128, 1>(m, f, (int)(ctas * (q.segs - 1)), s);
    trace_end(s);
    ++*launches;
    if (e != cudaSuccess) return e;
    trace_begin("decay_join", s);
    e = launch_pdl(decay_join_kernel, dim3((unsigned)((ctas * a.da * kN + 255) / 256)), dim3(256), 0, s, a, q.segs, q.seg_h,
                   static_cast<const float*>(q.seg_d));
    trace_end(s);
    ++*launches;
    if (e != cudaSuccess) return e;
  }
  trace_begin("decay_tc", s);
  const int blocks = (int)(ctas * q.segs);
  if (exact_state)
    e = a.da == 64 ? launch<64, 3>(m, q, blocks, s) : launch<128, 3>(m, q, blocks, s);
  else
    e = a.da == 64 ? launch<64, 1>(m, q, blocks, s) : launch<128, 1>(m, q, blocks, s);
  trace_end(s);
  ++*launches;
  return e;
}

cudaError_t launch_decay_pairs(const DecayPairs& a, cudaStream_t s, int* launches) {
  PairMaps m;
  PairParams p{};
  const int Hk = a.H / a.G;
  if (!rows_map(&m.q, a.q, a.B, a.H, a.L, a.dk, a.sq, &p.qn, &p.qh) ||
      !rows_map(&m.k, a.k, a.B, Hk, a.L, a.dk, a.sk, &p.kn, &p.kh) ||
      !rows_map(&m.v, a.v, a.B, Hk, a.L, a.dv, a.sv, &p.vn, &p.vh) ||
      !rows_map(&m.y, a.dy, a.B, a.H, a.L, a.dv, a.sy, &p.yn, &p.yh))
    return cudaErrorInvalidValue;
  p.B = a.B, p.H = a.H, p.L = a.L, p.G = a.G, p.lg = a.lg, p.sg = a.sg, p.count = a.count, p.scale = a.scale;
  p.row = a.row, p.col = a.col, p.status = a.status;
  trace_begin("decay_pairs", s);
  cudaError_t e;
  if (a.dk == 64)
    e = a.dv == 64 ? launch_pairs<64, 64>(m, p, s) : launch_pairs<64, 128>(m, p, s);
  else
    e = a.dv == 64 ? launch_pairs<128, 64>(m, p, s) : launch_pairs<128, 128>(m, p, s);
  trace_end(s);
  ++*launches;
  return e;
}

}  // namespace lz
