// k_decay_tc.cu -- one pass of the linear attention with a decay per head on the tensor cores (bf16),
// the state pass over segments of a long axis, and the products within a chunk that the gradient of
// log_decay needs.
//
// Chunks of 128 tokens, one after the other in the pass's direction; H the state that enters one:
//   S = A B^T,  P = S o D,  out = P C + from o (A H),  H' = all H + B^T (to o C)
// D the decays between the chunk's tokens, `from` and `to` those between a token and the chunk's edges.
// Every decay is a product of exponentials of sums of few log decays of one sign: for tokens of
// different 16-token blocks D = row (edge of its block to the one) G (blocks between) col, so that an
// element of P costs two multiplications instead of an exponential; within a block it is the exponential
// of a difference of two sums of at most 16.  A document's start counts as 2^-300, which is 0 in every
// product: no sum is infinite.
//
// A CTA takes 64 of C's channels of one head over the chunks of one segment; H stays in registers in
// fp32.  Twenty warps (five on each quarter of the SM, at 96 registers):
//   0      copies the tiles of A, B [128][da] and C [128][64] in by TMA, two stages ahead
//   1, 3   issue the MMAs: S and P C, and B^T C~ and A H
//   2      the decays of the next chunks
//   4-11   C~ = to o C in two or three bf16 parts (16 or 24 bits: the state is a sum over the whole
//          sequence, so its operands are not rounded), then P, rounded once to bf16, into TMEM
//   12-19  the state: H = all H + (B^T C~); its bf16 parts for the next chunk's A H (one part, as P is
//          rounded too, or three where the product with H itself is a result); then the rows of out
// TMEM: S 128 columns, P 64, B^T C~ 3 x 64 (its parts side by side: one reading of B for all of them),
// P C 64, A H 64.
//
// What bounds it is none of the peaks: 2 x 4096 tokens at 32 heads of 128 take 82 us, 3.0 TB/s and 38% of
// the tensor cycles, the shared memory about 80% busy with operands, copies and C~, the schedulers 56%.
// A chunk takes about 4400 cycles, of which each group of warps spends 900 instructions at four to five
// cycles; leaving out any one of the loads, of the MMAs, of P's or of out's arithmetic changes it by 5% at
// most, C~ by 15%.  What brought it there from 128 us: MMAs issued by a whole warp in uniform registers
// (a lane's branch: 90 cycles an MMA), loops kept short (instruction fetch was the first stall), out stored
// by whole sectors, scores of the next chunk ahead of P C.  Not kept: clusters of a head's two slices with
// multicast tiles (90 us), out through shared memory (148 us).
#include <math.h>

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
constexpr int kColS = 0, kColP = 128, kColKV = 192, kColY = 384, kColYs = 448;

enum {
  FA = 0, FB = 2, FC = 4, EA = 6, EB = 8, EC = 10,  // tiles full and empty, by stage
  FACF = 12, FACE = 14,                             // factors full and empty, by buffer
  CT = 16, KVR = 18, KVF = 20,                      // C~ ready, B^T C~ ready, read; by parity
  SR = 22, HR, HF, PR, YR, YF, FIX, DONE, DONE2, NB
};

// Of a chunk: row, log2 of the decay from the edge of a token's 16-token block to the token (from the
// block's start with it; with rev from behind it to the block's end), so that between two tokens of a
// block it is the difference; col the decays from a token to the other edge of its block; g those over
// the blocks between [the output's][the source's]; head and tail those over the blocks between the
// chunk's edge where the state enters (leaves) and a block.
struct alignas(16) Factors {
  float row[kC], col[kC];
  float g[64];
  float head[8], tail[8];
  float all;
};

struct Head {  // in front of the tiles
  Ctl<NB> ctl;
  Factors f[2];
};
constexpr int kHead = 3 * 1024;
static_assert(sizeof(Head) <= kHead, "barriers and factors");

template <int DA, int NPH>
struct Smem {
  static constexpr int kTile = kC * DA * 2;
  static constexpr int NA = 2, NBt = DA == 128 && NPH == 3 ? 1 : 2, NCt = 2;
  static constexpr int A = 0, B = A + NA * kTile, Ct = B + NBt * kTile, CP = Ct + NCt * kTileC;
  static constexpr int kPartH = DA * kN * 2;
  static constexpr int H = CP + 3 * kTileC;
  // a second place for the parts of C~ where there is no A (the state pass)
  static constexpr int CP2 = DA == 128 ? A : H + NPH * kPartH;
  static constexpr int kBytes = kHead + (DA == 128 ? H + NPH * kPartH : CP2 + 3 * kTileC);
  static_assert(DA != 128 || NA * kTile >= 3 * kTileC, "the second place lies over the tiles of A");
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

struct Maps {
  CUtensorMap a, b, c;
};

struct TcParams {
  DecayPass p;
  int an, ah, bn, bh, cn, ch;  // 0 where a tensor repeats over sequences or heads, else 1
  int parts;                   // bf16 parts of C~
  float log_scale;             // log2 of what P is scaled by
  DecaySegs g;
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// Operand descriptors of 128-byte-swizzled tiles differ in their lower words only: the address, and the
// distance of 64-column blocks (K-major operands do not use it).  A k-step of 16 adds to the lower word.
constexpr uint32_t kDescUpper = (1024u >> 4) | (1u << 14) | (kSw128 << 29);
__device__ __forceinline__ uint32_t desc_lower(uint32_t saddr, uint32_t block) { return (saddr >> 4) | ((block >> 4) << 16); }
__host__ __device__ constexpr uint32_t step_k(int j) { return (uint32_t)(j >> 2) * (kC * 128 / 16) + (uint32_t)(j & 3) * 2; }
__host__ __device__ constexpr uint32_t step_mn(int j) { return (uint32_t)j * (16 * 128 / 16); }

// D(tmem) (+)= A(smem) * B(smem)^T, and with A in TMEM.  The whole warp calls and one lane issues, so
// that addresses and descriptors stay in uniform registers: from a branch that one lane takes, each MMA
// cost about 90 cycles of moves.
__device__ __forceinline__ void mma_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\telect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescUpper), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_lo_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\telect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescUpper), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// elect.sync picks the same lane each time, whose MMAs these are.
__device__ __forceinline__ void commit_lo(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// wait_bar with its polling out of line: the roles' loops are long, and what they share should be in the
// instruction cache once.
template <int N>
__device__ __noinline__ bool wait_polls(Ctl<N>* ctl, int i, uint32_t parity) {
  return wait_bar(ctl, i, parity);
}
template <int N>
__device__ __forceinline__ bool wait_for(Ctl<N>* ctl, int i, uint32_t parity) {
  return mbar_try_wait(&ctl->bar[i], parity) || wait_polls(ctl, i, parity);
}
// A wait by a whole warp with one answer.
template <int N>
__device__ __forceinline__ bool wait_warp(Ctl<N>* ctl, int i, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_for(ctl, i, parity));
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ float f32(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// The upper halves of two words, the first's below: two floats cut to bf16.
__device__ __forceinline__ uint32_t upper(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float2 cut(float2 v) {
  return make_float2(f32(__float_as_uint(v.x) & 0xffff0000u), f32(__float_as_uint(v.y) & 0xffff0000u));
}
// Two values as sums of bf16 parts.  Three parts of 8 bits are the whole 24: cut off, the rest is exact
// each time.  Two: the second is rounded to nearest.
__device__ __forceinline__ void split(float2 v, bool three, uint32_t (&o)[3]) {
  const float2 minus = make_float2(-1.f, -1.f);
  o[0] = upper(v.x, v.y);
  v = f2_fma(cut(v), minus, v);
  if (three) {
    o[1] = upper(v.x, v.y);
    v = f2_fma(cut(v), minus, v);
    o[2] = upper(v.x, v.y);
  } else {
    o[1] = pack_bf16x2(v.x, v.y);
  }
}

// One warp: the factors of a chunk from its log2 decays, four tokens a lane, four lanes a block; a lane's share is made in registers, then stored.
struct Share {
  float x[4], row[4], col[4], g[2], head, tail, all;
  __device__ __forceinline__ void make(bool rev) {
    const int lane = threadIdx.x & 31, own = lane >> 2;
    float pre[4], suf[4];
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
    float sum = 0.f, first = 0.f, last = 0.f, between[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = __shfl_sync(0xffffffffu, up, 4 * j + 3);
      if (j < own) first += t;
      if (j > own) last += t;
      sum += t;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int a = (lane >> 3) + 4 * e, b = lane & 7;
        if (j > min(a, b) && j < max(a, b)) between[e] += t;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float p = pre[k] + before, s = suf[k] + behind;
      row[k] = rev ? s : p, col[k] = exp2f(rev ? p : s);
    }
    g[0] = exp2f(between[0]), g[1] = exp2f(between[1]);
    head = exp2f(rev ? last : first), tail = exp2f(rev ? first : last), all = exp2f(sum);
  }
  __device__ __forceinline__ void put(Factors& f) const {
    const int lane = threadIdx.x & 31;
    *reinterpret_cast<float4*>(f.row + 4 * lane) = make_float4(row[0], row[1], row[2], row[3]);
    *reinterpret_cast<float4*>(f.col + 4 * lane) = make_float4(col[0], col[1], col[2], col[3]);
    f.g[lane] = g[0], f.g[lane + 32] = g[1];
    if ((lane & 3) == 0) f.head[lane >> 2] = head, f.tail[lane >> 2] = tail;
    if (lane == 0) f.all = all;
  }
};

// Four of a chunk's log decays in log2 (a lane's own); past the sequence's end 0.
__device__ __forceinline__ void load_decays(const float* lg, int64_t st, int t0, int count, float (&x)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = t0 + 4 * lane + k;
    const float g = t < count ? lg[t * st] : 0.f;
    x[k] = g < kDecayNone ? -300.f : g * 1.4426950408889634f;
  }
}

// A block's 16 numbers.
__device__ __forceinline__ void block_of(const float* x, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 q = *reinterpret_cast<const float4*>(x + 4 * j);
    v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
  }
}

// The decays within a 16-token block between token `o` of it and each token s <= o and 0 elsewhere, by running
// sums; x: the block's log2 decays.
__device__ __forceinline__ void block_decays(const float* x, int o, float (&d)[16]) {
  float v[16];
  block_of(x, v);
  float sum = 0.f;
#pragma unroll
  for (int s = 15; s >= 0; --s) {
    sum = s >= o ? 0.f : sum + v[s < 15 ? s + 1 : 15];
    d[s] = s > o ? 0.f : ex2_approx(sum);
  }
}

// A warp's 32 rows from token t0 on, 64 bytes of each lane's row: four neighbouring lanes exchange their
// pieces of 16 and store each row's together (whole sectors, and a quarter of the lines a store).  Rows
// from L on are not there.
__device__ __forceinline__ void put64(unsigned char* out, int64_t pitch, int t0, int L, uint4 (&c)[4]) {
  const int lane = threadIdx.x & 31;
  auto swap = [&](uint4& lower, uint4& upper, int bit) {
    const bool up = lane & bit;
    uint4 t = up ? lower : upper;
    t.x = __shfl_xor_sync(0xffffffffu, t.x, bit), t.y = __shfl_xor_sync(0xffffffffu, t.y, bit);
    t.z = __shfl_xor_sync(0xffffffffu, t.z, bit), t.w = __shfl_xor_sync(0xffffffffu, t.w, bit);
    if (up) lower = t;
    else upper = t;
  };
  swap(c[0], c[1], 1), swap(c[2], c[3], 1);
  swap(c[0], c[2], 2), swap(c[1], c[3], 2);
  const int t = t0 + (lane & ~3);
  unsigned char* o = out + t * pitch + (lane & 3) * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k, o += pitch)
    if (t + k < L) *reinterpret_cast<uint4*>(o) = c[k];
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
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
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
    for (int i = 0; i < NB; ++i) {
      const bool both = i == FACE || i == FACE + 1, score = i == CT || i == CT + 1 || i == PR || i == FIX,
                 state = i == KVF || i == KVF + 1 || i == HR || i == YF;
      // the tiles of A and B are read by both MMA warps
      const bool shared = (i >= EA && i < EC) && !q.g.states_only;
      mbar_init(&ctl->bar[i], both ? kScoreWarps + kStateWarps : score ? kScoreWarps : state ? kStateWarps : shared ? 2 : 1);
    }
    ctl->abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
  pdl_wait();

  int count = p.L;
  if (p.count) {
    count = p.count[n];
    if (count < 0 || count > p.L) {
      if (tid == 0) raise_status(p.status, kDevCheck);
      count = 0;
    }
  }
  count = __shfl_sync(0xffffffffu, count, 0);  // (known to be the same in the warp)
  // this segment's chunks, in the pass's order from `first` on
  const int chunks = (count + kC - 1) / kC;
  const int done = min(seg * q.g.cps, chunks), num = min(q.g.cps, chunks - done);
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
        const int t0 = token(it), sb = it % Sm::NBt, sa = it % Sm::NA;
        const int sc = it % Sm::NCt;
        // in the order in which the stages come free
        if (it >= Sm::NBt && !(ok = wait_for(ctl, EB + sb, (it / Sm::NBt - 1) & 1))) break;
        mbar_arrive_expect_tx(&ctl->bar[FB + sb], Sm::kTile);
#pragma unroll
        for (int k = 0; k < DA / 64; ++k)
          tma_load_4d(sm + Sm::B + sb * Sm::kTile + k * (kC * 128), &maps.b, 64 * k, t0, hb, nb, &ctl->bar[FB + sb]);
        armed_b[0] += sb == 0, armed_b[1] += sb == 1;
        if (!q.g.states_only) {
          if (it >= Sm::NA && !(ok = wait_for(ctl, EA + sa, (it / Sm::NA - 1) & 1))) break;
          mbar_arrive_expect_tx(&ctl->bar[FA + sa], Sm::kTile);
#pragma unroll
          for (int k = 0; k < DA / 64; ++k)
            tma_load_4d(sm + Sm::A + sa * Sm::kTile + k * (kC * 128), &maps.a, 64 * k, t0, ha, na, &ctl->bar[FA + sa]);
          armed_a[0] += sa == 0, armed_a[1] += sa == 1;
        }
        if (it >= Sm::NCt && !(ok = wait_for(ctl, EC + sc, (it / Sm::NCt - 1) & 1))) break;
        mbar_arrive_expect_tx(&ctl->bar[FC + sc], kTileC);
        tma_load_4d(sm + Sm::Ct + sc * kTileC, &maps.c, c0, t0, hc, nc, &ctl->bar[FC + sc]);
        armed_c[0] += sc == 0, armed_c[1] += sc == 1;
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
    if (!q.g.states_only) {
      const uint32_t sb = smem_u32(sm);
      const uint32_t id_s = idesc_bf16(kC, kC, false, false), id_c = idesc_bf16(kC, kN, false, true);
      const uint32_t da = desc_lower(sb + Sm::A, 16), db = desc_lower(sb + Sm::B, 16), dc = desc_lower(sb + Sm::Ct, kC * 128);
      auto scores = [&](int it) {  // S = A B^T
        if (!wait_warp(ctl, FB + it % Sm::NBt, (it / Sm::NBt) & 1) || !wait_warp(ctl, FA + it % Sm::NA, (it / Sm::NA) & 1))
          return false;
        if (ragged(it) && !wait_warp(ctl, FIX, 0)) return false;
        tc_fence_after();
        const uint32_t a = da + it % Sm::NA * (Sm::kTile / 16), b = db + it % Sm::NBt * (Sm::kTile / 16);
#pragma unroll 4
        for (int j = 0; j < DA / 16; ++j) mma_lo(tmem + kColS, a + step_k(j), b + step_k(j), id_s, j > 0);
        commit_lo(&ctl->bar[SR]);
        commit_lo(&ctl->bar[EA + it % Sm::NA]);
        commit_lo(&ctl->bar[EB + it % Sm::NBt]);
        return true;
      };
      bool ok = num == 0 || scores(0);
#pragma unroll 1
      for (int it = 0; it < num && ok; ++it) {
        // P is there, so S has been read: the next scores first, which are waited for sooner than P C
        if (!(ok = wait_warp(ctl, PR, it & 1))) break;
        if (it + 1 < num && !(ok = scores(it + 1))) break;
        if (it > 0 && !(ok = wait_warp(ctl, YF, (it - 1) & 1))) break;
        tc_fence_after();
        const uint32_t c = dc + it % Sm::NCt * (kTileC / 16);
#pragma unroll 4
        for (int j = 0; j < kC / 16; ++j) mma_lo_ts(tmem + kColY, tmem + kColP + 8 * j, c + step_mn(j), id_c, j > 0);
        commit_lo(&ctl->bar[YR]);
        commit_lo(&ctl->bar[EC + it % Sm::NCt]);
      }
      if (!ok) ctl->abort = 1;
      commit_lo(&ctl->bar[DONE]);
      drain_bar(ctl, DONE, 1, globaltimer_ns());
      __syncwarp();
    }
  } else if (warp == 3) {
    const uint32_t sb = smem_u32(sm);
    constexpr uint32_t kRow = kC * 128;  // bytes of a 64-column block of a tile
    static_assert(kN == kDecaySlice, "segments' states are kept by slices");
    static_assert(kRow == kTileC, "the parts of C~ are the blocks of one operand");
    const uint32_t id_kv = idesc_bf16(128, q.parts * kN, true, true), id_h = idesc_bf16(kC, kN, false, true);
    const uint32_t da = desc_lower(sb + Sm::A, 16), db = desc_lower(sb + Sm::B, kRow), dp = desc_lower(sb + Sm::CP, kRow),
                   dp2 = desc_lower(sb + Sm::CP2, kRow), dh = desc_lower(sb + Sm::H, kRow);
    bool ok = true;
#pragma unroll 1
    for (int it = 0; it < num && ok; ++it) {
      // B^T C~, into alternate columns where there are no scores
      const bool other = q.g.states_only && (it & 1);
      const int lag = q.g.states_only ? 2 : 1;
      if (!(ok = wait_warp(ctl, FB + it % Sm::NBt, (it / Sm::NBt) & 1))) break;
      if (!(ok = wait_warp(ctl, CT + (it & 1), (it >> 1) & 1))) break;
      if (it >= lag && !(ok = wait_warp(ctl, KVF + ((it - lag) & 1), ((it - lag) >> 1) & 1))) break;
      tc_fence_after();
      const uint32_t b = db + it % Sm::NBt * (Sm::kTile / 16);
#pragma unroll 4
      for (int j = 0; j < kC / 16; ++j)
        mma_lo(tmem + (other ? 0 : kColKV), b + step_mn(j), (other ? dp2 : dp) + step_mn(j), id_kv, j > 0);
      commit_lo(&ctl->bar[KVR + (it & 1)]);
      commit_lo(&ctl->bar[EB + it % Sm::NBt]);
      if (q.g.states_only) {
        commit_lo(&ctl->bar[EC + it % Sm::NCt]);
        continue;
      }
      // A H, the smallest parts first, while the sum and what its additions cut off are small
      if (!(ok = wait_warp(ctl, HR, it & 1))) break;
      if (!(ok = wait_warp(ctl, FA + it % Sm::NA, (it / Sm::NA) & 1))) break;
      if (it > 0 && !(ok = wait_warp(ctl, YF, (it - 1) & 1))) break;
      tc_fence_after();
      const uint32_t a = da + it % Sm::NA * (Sm::kTile / 16);
#pragma unroll 1
      for (int k = NPH - 1; k >= 0; --k)
#pragma unroll 4
        for (int j = 0; j < DA / 16; ++j)
          mma_lo(tmem + kColYs, a + step_k(j), dh + k * (Sm::kPartH / 16) + step_mn(j), id_h, k < NPH - 1 || j > 0);
      commit_lo(&ctl->bar[HF]);
      commit_lo(&ctl->bar[EA + it % Sm::NA]);
    }
    if (!ok) ctl->abort = 1;
    commit_lo(&ctl->bar[DONE2]);
    drain_bar(ctl, DONE2, 1, globaltimer_ns());
    __syncwarp();
  } else if (warp == 2) {
    const float* lg = p.lg + n * p.sg.n + h * p.sg.h;
    Share f;
    if (num > 0) load_decays(lg, p.sg.t, token(0), count, f.x);
    bool ok = true;
#pragma unroll 1
    for (int it = 0; it < num && ok; ++it) {
      float next[4] = {};
      if (it + 1 < num) load_decays(lg, p.sg.t, token(it + 1), count, next);
      f.make(p.rev);
      if (it > 1 && !(ok = wait_for(ctl, FACE + (it & 1), (it / 2 - 1) & 1))) break;
      f.put(hd.f[it & 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[FACF + (it & 1)]);
#pragma unroll
      for (int k = 0; k < 4; ++k) f.x[k] = next[k];
    }
    if (!ok) ctl->abort = 1;
  } else if (warp >= 4 && warp < 12) {
    const int half = (warp - 4) >> 2, qw = warp & 3, wt = tid - 128;  // thread of the group
    const int o = 32 * qw + lane, I = o >> 4;
    const uint32_t tl = (uint32_t)(qw * 32) << 16;
    // Of the 16-token blocks of sources, a warp's rows see `full` ones wholly, from `j0` on every other
    // one (its half of them), and take part in two, of which it has j1: the decays within a block for
    // the rows that lie in it, for the others all of it or nothing.  The rest of P is always 0.
    const int full = p.rev ? 3 - qw : qw, j0 = p.rev ? 2 * qw + 2 + half : half, j1 = 2 * qw + half;
    const bool own = (lane >> 4) == half, sees = p.rev ? half == 1 : half == 0;
    if (!q.g.states_only) {
      const uint32_t z[8] = {};
      for (int j = half; j < 8; j += 2)
        if (p.rev ? j < 2 * qw : j > 2 * qw + 1) tmem_st8(tmem + tl + kColP + 8 * j, z);
      tmem_st_wait();
    }
    bool ok = true;
#pragma unroll 1
    for (int it = 0; it < num && ok; ++it) {
      const int valid = min(kC, count - token(it));
      unsigned char* tc_ = sm + Sm::Ct + it % Sm::NCt * kTileC;
      if (!(ok = wait_for(ctl, FC + it % Sm::NCt, (it / Sm::NCt) & 1))) break;
      if (ragged(it)) {
        if (!(ok = wait_for(ctl, FB + it % Sm::NBt, (it / Sm::NBt) & 1))) break;
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
      if (!(ok = wait_for(ctl, FACF + (it & 1), (it >> 1) & 1))) break;
      const Factors& f = hd.f[it & 1];
      // C~ (its tiles are free once the chunk before has been multiplied; with two places the one before it)
      const int lag = q.g.states_only ? 2 : 1;
      if (it >= lag && !(ok = wait_for(ctl, KVR + ((it - lag) & 1), ((it - lag) >> 1) & 1))) break;
      unsigned char* cp = sm + (q.g.states_only && (it & 1) ? Sm::CP2 : Sm::CP);
#pragma unroll 2
      for (int e = 0; e < kTileC / 16 / (32 * kScoreWarps); ++e) {
        const int at = (wt + 32 * kScoreWarps * e) * 16;  // byte of the tile: the swizzle stays as it is
        const float w = f.col[at >> 7] * f.tail[at >> 11] * p.scale_in;
        const float2 w2 = make_float2(w, w);
        const uint4 v = *reinterpret_cast<const uint4*>(tc_ + at);
        const bool three = q.parts > 2;
        uint32_t o0[3], o1[3], o2[3], o3[3];
        split(f2_mul(w2, make_float2(lo_f(v.x), hi_f(v.x))), three, o0);
        split(f2_mul(w2, make_float2(lo_f(v.y), hi_f(v.y))), three, o1);
        split(f2_mul(w2, make_float2(lo_f(v.z), hi_f(v.z))), three, o2);
        split(f2_mul(w2, make_float2(lo_f(v.w), hi_f(v.w))), three, o3);
        unsigned char* d = cp + at;
        *reinterpret_cast<uint4*>(d) = make_uint4(o0[0], o1[0], o2[0], o3[0]);
        *reinterpret_cast<uint4*>(d + kTileC) = make_uint4(o0[1], o1[1], o2[1], o3[1]);
        if (three) *reinterpret_cast<uint4*>(d + 2 * kTileC) = make_uint4(o0[2], o1[2], o2[2], o3[2]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[CT + (it & 1)]);
      if (q.g.states_only) {
        if (lane == 0) mbar_arrive(&ctl->bar[FACE + (it & 1)]);
        continue;
      }
      // P, 16 columns at a time
      const float row = f.row[o] + q.log_scale, rf = ex2_approx(row);
      const uint32_t ts = tmem + tl + kColS, tp = tmem + tl + kColP;
      float d[16];
      block_of((own ? f.row : f.col) + 16 * j1, d);
      const int io = lane & 15;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float e = (p.rev ? k >= io : k <= io) ? ex2_approx(row - d[k]) : 0.f;
        d[k] = own ? e : sees ? rf * d[k] : 0.f;
      }
      if (!(ok = wait_warp(ctl, SR, it & 1))) break;
      if (it > 0 && !(ok = wait_warp(ctl, YR, (it - 1) & 1))) break;  // the chunk before has been multiplied
      tc_fence_after();
      {
        uint32_t s[16], w[8];
        tmem_ld16(ts + 16 * j1, s);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 u = f2_mul(make_float2(f32(s[2 * k]), f32(s[2 * k + 1])), make_float2(d[2 * k], d[2 * k + 1]));
          w[k] = pack_bf16x2(u.x, u.y);
        }
        tmem_st8(tp + 8 * j1, w);
      }
#pragma unroll 1
      for (int k = 0; k < full; ++k) {
        const int j = j0 + 2 * k;
        uint32_t s[16], w[8];
        tmem_ld16(ts + 16 * j, s);
        const float r1 = rf * f.g[I * 8 + j];
        const float2 r = make_float2(r1, r1);
        float2 c[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v = *reinterpret_cast<const float4*>(&f.col[16 * j + 4 * e]);
          c[2 * e] = f2_mul(r, make_float2(v.x, v.y)), c[2 * e + 1] = f2_mul(r, make_float2(v.z, v.w));
        }
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 u = f2_mul(make_float2(f32(s[2 * e]), f32(s[2 * e + 1])), c[e]);
          w[e] = pack_bf16x2(u.x, u.y);
        }
        tmem_st8(tp + 8 * j, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[PR]), mbar_arrive(&ctl->bar[FACE + (it & 1)]);
    }
    if (!ok) ctl->abort = 1;
  } else if (warp >= 12 && warp < 20) {
    const int half = (warp - 12) >> 2, qw = warp & 3;
    const int i = 32 * qw + lane;  // row of the state, row of the output
    const bool mine = i < DA;
    const uint32_t tl = tmem + ((uint32_t)(qw * 32) << 16) + 32 * half;
    float x[32];
    // this thread's columns in a state of the caller's
    const int c1 = c0 + 32 * half, state_step = p.state_t ? DA : 1;
    const int64_t state_at = (int64_t)unit * DA * p.dc + (p.state_t ? c1 * DA + i : i * p.dc + c1);
    float* seg_h = q.g.seg_h + ((((int64_t)seg * units + unit) * slices + slice) * DA + i) * kN + 32 * half;
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = 0.f;
    if (mine && !q.g.states_only) {
      if (q.g.segs > 1) {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = seg_h[j];
      } else if (p.init) {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = p.init[state_at + j * state_step];
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
              split(make_float2(x[8 * j + 2 * k], x[8 * j + 2 * k + 1]), true, o[k]);
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
    if (num > 0 && !q.g.states_only) put_state();
#pragma unroll 1
    for (int it = 0; it < num && ok; ++it) {
      if (!(ok = wait_for(ctl, FACF + (it & 1), (it >> 1) & 1))) break;
      const Factors& f = hd.f[it & 1];
      const float from = exp2f(f.row[i]) * f.head[i >> 4] * p.scale_out, all = f.all;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[FACE + (it & 1)]);
      product *= all;
      if (NPH == 3 && p.edge) {
        // the states at the chunks' edges, for the gradient of log_decay: this thread's 8 x 4 of each, a warp's
        // side by side (2 x 4096 tokens, 32 heads of 128: 134 MB, a pass 121 -> 137 us)
        const int64_t at = ((int64_t)unit * ((p.L + kC - 1) / kC) + first + dir * it) * slices + slice;
        float4* e = reinterpret_cast<float4*>(p.edge) + at * (DA * kN / 4) + 8 * half * DA + i;
        if (p.through) {
          // what passes over the whole chunk: decayed, <H, the state that enters from the other side>
          float2 s2 = make_float2(0.f, 0.f);
          if (mine) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 v = e[j * DA];
              s2 = f2_fma(make_float2(x[4 * j], x[4 * j + 1]), make_float2(v.x, v.y), s2);
              s2 = f2_fma(make_float2(x[4 * j + 2], x[4 * j + 3]), make_float2(v.z, v.w), s2);
            }
          }
          const float s = warp_sum(s2.x + s2.y);
          if (lane == 0) p.through[at * kDecayEdgeWarps + 4 * half + qw] = all * s;
          // the next chunk's into L2, a line a thread (the passes 366 -> 359 us)
          if (it + 1 < num && 128 * half + i < DA * kN / 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<float4*>(p.edge) + (at + slices) * (DA * kN / 4) + 8 * (128 * half + i)));
        } else if (mine) {
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j * DA] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        }
      }
      // H = all H + B^T C~, whose parts are added up from the smallest
      if (!(ok = wait_for(ctl, KVR + (it & 1), (it >> 1) & 1))) break;
      tc_fence_after();
      const uint32_t tk = tl + (q.g.states_only && (it & 1) ? 0 : kColKV);
      const float2 all2 = make_float2(all, all);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t k0[8], k1[8], k2[8] = {};
        tmem_ld8(tk + 8 * e, k0);
        tmem_ld8(tk + kN + 8 * e, k1);
        if (q.parts > 2) tmem_ld8(tk + 2 * kN + 8 * e, k2);
        tmem_ld_wait();
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
          float* h2 = &x[8 * e + 2 * j];
          const float2 v = f2_add(make_float2(f32(k2[2 * j]), f32(k2[2 * j + 1])), make_float2(f32(k1[2 * j]), f32(k1[2 * j + 1])));
          const float2 w = f2_add(v, make_float2(f32(k0[2 * j]), f32(k0[2 * j + 1])));
          const float2 u = f2_fma(all2, make_float2(h2[0], h2[1]), w);
          h2[0] = u.x, h2[1] = u.y;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[KVF + (it & 1)]);
      if (q.g.states_only) continue;
      if (!(ok = wait_for(ctl, HF, it & 1))) break;
      if (it + 1 < num) put_state();
      // out = P C + from o (A H)
      const int t = token(it) + i;
      const bool live = t < count;
      if (!(ok = wait_for(ctl, YR, it & 1))) break;
      tc_fence_after();
      float d = 0.f;
      uint4 w[4];
      const float2 from2 = make_float2(from, from);
      const bool tail = ragged(it);
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
        if (NPH == 3 && px && live) {
          const uint4* xr = reinterpret_cast<const uint4*>(px + t * p.sx.t + 16 * e);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 u = xr[k];
            const uint32_t z[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              d = fmaf(lo_f(z[r]), f32(ys[8 * k + 2 * r]), d);
              d = fmaf(hi_f(z[r]), f32(ys[8 * k + 2 * r + 1]), d);
            }
          }
        }
        float2 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = f2_fma(from2, make_float2(f32(ys[2 * j]), f32(ys[2 * j + 1])), make_float2(f32(y[2 * j]), f32(y[2 * j + 1])));
          if (tail && !live) v[j] = make_float2(0.f, 0.f);  // rows behind the sequence may have held anything
        }
        if (p.out_f32) {
          unsigned char* o = static_cast<unsigned char*>(p.out) + (so + 16 * e) * 4;
          auto bits = [&](int j) {
            return make_uint4(__float_as_uint(v[j].x), __float_as_uint(v[j].y), __float_as_uint(v[j + 1].x), __float_as_uint(v[j + 1].y));
          };
          uint4 c[4] = {bits(0), bits(2), bits(4), bits(6)};
          put64(o, p.so.t * 4, t - lane, p.L, c);
        } else {
          auto bits = [&](int j) {
            return make_uint4(pack_bf16x2(v[j].x, v[j].y), pack_bf16x2(v[j + 1].x, v[j + 1].y), pack_bf16x2(v[j + 2].x, v[j + 2].y),
                              pack_bf16x2(v[j + 3].x, v[j + 3].y));
          };
          if (e == 0)
            w[0] = bits(0), w[1] = bits(4);
          else
            w[2] = bits(0), w[3] = bits(4);
        }
      }
      if (!p.out_f32) put64(static_cast<unsigned char*>(p.out) + so * 2, p.so.t * 2, t - lane, p.L, w);
      if (NPH == 3 && px && live) dot[t] = from * d;
    }
    if (!ok) ctl->abort = 1;
    if (ok && q.g.states_only) {
      if (mine) {
#pragma unroll
        for (int j = 0; j < 32; ++j) seg_h[j] = x[j];
      }
      if (i == 0 && half == 0) q.g.seg_d[((int64_t)seg * units + unit) * slices + slice] = product;
    } else if (ok) {
      if (mine && p.fin && seg == q.g.segs - 1) {
#pragma unroll
        for (int j = 0; j < 32; ++j) p.fin[state_at + j * state_step] = x[j];
      }
      // the rows of whole chunks behind the sequence
      const int all_chunks = (p.L + kC - 1) / kC;
      const int za = max(seg * q.g.cps, chunks), zb = min((seg + 1) * q.g.cps, all_chunks);
      const int es = p.out_f32 ? 4 : 2;
      for (int c = za; c < zb; ++c)
        for (int b = 0; b < es / 2; ++b) {
          uint4 z[4] = {};
          put64(static_cast<unsigned char*>(p.out) + so * es + 64 * b, p.so.t * es, c * kC + 32 * qw, p.L, z);
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

// ---------------------------------------------------------------------------------
// Within a chunk: inside_t = sum_{s < t <= i} W_is, W_is = scale (q_i . k_s) D (dy_i . v_s), from exact products
// of the bf16 rows in fp32 sums: of those products alone that pass over t, since a difference of whole rows
// and columns would leave the rounding of all others.  Two CTAs an SM, each chunk after chunk: the two scores by
// MMAs (dy takes q's place in shared memory once the first is done; the next chunk's rows come while this
// one's are summed), then eight warps of which each has every other 32 columns of its 32 rows: a thread makes
// the running sums of its row, E_it = sum_{s < t} W_is from the 32 columns' first on, and those of the rows
// from t on are summed over the warp by halving exchanges.  The last step adds, for the columns of a group, the
// whole groups before it: of the rows of later groups as one number each (all), of its own rows those from t on
// (rows).  (64 heads x 4096 tokens of 128: 55 us; with whole rows and columns 52, and a CTA a chunk 62.)
// ---------------------------------------------------------------------------------
constexpr int kPairThreads = 384;
enum { GQ = 0, GY, GS, GP, GR, GF = 5, GE = 7, GN = 9 };  // GF, GE: by parity
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
  float* inside;  // [B,H,L]
  unsigned* status;
};
struct alignas(16) PairHead {
  Ctl<GN> ctl;
  Factors f[2];
  float x[2][kC];
  // [parity][half of the columns, or quarter of the rows]
  float rows[2][2][kC], cols[2][4][kC];
  float all[2][4][4];  // [parity][quarter of the rows][of the columns, before the rows' own]
};
template <int DK, int DV>
struct PairSmem {
  static constexpr int kHead = 11264;
  static_assert(sizeof(PairHead) <= kHead, "barriers, factors and sums");
  static constexpr int kQ = kC * DK * 2, kV = kC * DV * 2, kFirst = kQ > kV ? kQ : kV;
  static constexpr int Q = 0, K = kFirst, V = K + kQ, kBytes = kHead + V + kV;
};

// 32 values a lane, of 32 columns: lane j gets the sum over the lanes of column j, in a fixed order.
__device__ __forceinline__ float column_sums(float (&w)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < o) w[j] = (up ? w[j + o] : w[j]) + __shfl_xor_sync(0xffffffffu, up ? w[j] : w[j + o], o);
  }
  return w[0];
}

template <int DK, int DV>
__global__ void __launch_bounds__(kPairThreads, 2)
    decay_pairs_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams p, int chunks, int items) {
  using Sm = PairSmem<DK, DV>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  PairHead& hd = *reinterpret_cast<PairHead*>(smem_raw);
  Ctl<GN>* ctl = &hd.ctl;
  unsigned char* sm = smem_raw + Sm::kHead;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (tid == 0) raise_status(p.status, kDevCheck);
    return;
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem, 256);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < GN; ++i) mbar_init(&ctl->bar[i], i == GR || i >= GE ? 8 : 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
  pdl_wait();
  // item w: chunk w mod chunks of head w / chunks; those behind a sequence's end are nobody's
  struct Item {
    int unit, n, h, t0, count;
  };
  auto item_of = [&](int w) {
    Item i;
    i.unit = w / chunks, i.t0 = (w - i.unit * chunks) * kC;
    i.n = i.unit / p.H, i.h = i.unit - i.n * p.H;
    i.count = p.count ? p.count[i.n] : p.L;
    if (i.count < 0 || i.count > p.L) i.count = 0;  // flagged by the passes
    i.count = __shfl_sync(0xffffffffu, i.count, 0);
    return i;
  };
  bool ok = true;
  int it = 0;  // items done
  if (warp == 0) {
#pragma unroll 1
    for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
      const Item i = item_of(w);
      if (i.t0 >= i.count) continue;
      // the last item's rows have been multiplied
      if (it > 0 && !(ok = wait_warp(ctl, GP, (it - 1) & 1))) break;
      const int hk = i.h / p.G;
      if (lane == 0) {
        mbar_arrive_expect_tx(&ctl->bar[GQ], 2 * Sm::kQ);
#pragma unroll
        for (int k = 0; k < DK / 64; ++k) {
          tma_load_4d(sm + Sm::Q + k * kC * 128, &maps.q, 64 * k, i.t0, p.qh * i.h, p.qn * i.n, &ctl->bar[GQ]);
          tma_load_4d(sm + Sm::K + k * kC * 128, &maps.k, 64 * k, i.t0, p.kh * hk, p.kn * i.n, &ctl->bar[GQ]);
        }
        mbar_arrive_expect_tx(&ctl->bar[GY], 2 * Sm::kV);
#pragma unroll
        for (int k = 0; k < DV / 64; ++k)
          tma_load_4d(sm + Sm::V + k * kC * 128, &maps.v, 64 * k, i.t0, p.vh * hk, p.vn * i.n, &ctl->bar[GY]);
      }
      __syncwarp();
      ++it;
      if (!(ok = wait_warp(ctl, GS, (it - 1) & 1))) break;
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < DV / 64; ++k)
          tma_load_4d(sm + Sm::Q + k * kC * 128, &maps.y, 64 * k, i.t0, p.yh * i.h, p.yn * i.n, &ctl->bar[GY]);
      }
      __syncwarp();
    }
    if (!ok) ctl->abort = 1;
    const uint64_t began = globaltimer_ns();
    drain_bar(ctl, GQ, it, began);
    drain_bar(ctl, GY, it, began);
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t sb = smem_u32(sm), id = idesc_bf16(kC, kC, false, false);
    const uint32_t dq = desc_lower(sb + Sm::Q, 16), dk = desc_lower(sb + Sm::K, 16), dv = desc_lower(sb + Sm::V, 16);
#pragma unroll 1
    for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
      const Item i = item_of(w);
      if (i.t0 >= i.count) continue;
      if (!(ok = wait_warp(ctl, GQ, it & 1))) break;
      if (it > 0 && !(ok = wait_warp(ctl, GE + ((it - 1) & 1), ((it - 1) >> 1) & 1))) break;  // the last scores are read
      tc_fence_after();
#pragma unroll 4
      for (int j = 0; j < DK / 16; ++j) mma_lo(tmem, dq + step_k(j), dk + step_k(j), id, j > 0);
      commit_lo(&ctl->bar[GS]);
      if (!(ok = wait_warp(ctl, GY, it & 1))) break;
      tc_fence_after();
#pragma unroll 4
      for (int j = 0; j < DV / 16; ++j) mma_lo(tmem + 128, dq + step_k(j), dv + step_k(j), id, j > 0);
      commit_lo(&ctl->bar[GP]);
      ++it;
    }
    if (!ok) ctl->abort = 1;
    // what was issued has ended: the last item's products, or the one broken off
    if (!ok) commit_lo(&ctl->bar[GP]);
    drain_bar(ctl, GP, it + (ok ? 0 : 1), globaltimer_ns());
    __syncwarp();
  } else if (warp == 2) {
#pragma unroll 1
    for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
      const Item i = item_of(w);
      if (i.t0 >= i.count) continue;
      Share v;
      load_decays(p.lg + i.n * p.sg.n + i.h * p.sg.h, p.sg.t, i.t0, i.count, v.x);
      v.make(false);
      const int par = it & 1;
      if (it > 1 && !(ok = wait_warp(ctl, GE + par, ((it >> 1) - 1) & 1))) break;
      *reinterpret_cast<float4*>(hd.x[par] + 4 * lane) = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
      v.put(hd.f[par]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[GF + par]);
      ++it;
    }
    if (!ok) ctl->abort = 1;
  } else if (warp >= 4) {
    const int half = (warp - 4) >> 2, qw = warp & 3, o = 32 * qw + lane, I = o >> 4;
    const uint32_t tl = tmem + ((uint32_t)(qw * 32) << 16);
#pragma unroll 1
    for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
      const Item i = item_of(w);
      if (i.t0 >= i.count) continue;
      const int par = it & 1;
      if (!(ok = wait_warp(ctl, GF + par, (it >> 1) & 1))) break;
      if (!(ok = wait_warp(ctl, GP, it & 1))) break;
      tc_fence_after();
      const Factors& f = hd.f[par];
      const float rf = exp2f(f.row[o]);
      const bool there = i.t0 + o < i.count;
      float sum = 0.f;
#pragma unroll 1
      for (int g = half; g <= qw; g += 2) {
        uint32_t s[32];
        float z[32];
        if (g == qw) {
          // the thread's own block of 16 by running sums, the one before it wholly, what is behind nothing
          float d[16];
          block_decays(hd.x[par] + 16 * I, lane & 15, d);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float in = j == (lane & 15) ? 0.f : d[j];
            z[j] = lane < 16 ? in : rf * f.col[32 * g + j];
            z[16 + j] = lane < 16 ? 0.f : in;
          }
        } else {
          const float r0 = rf * f.g[I * 8 + 2 * g], r1 = rf * f.g[I * 8 + 2 * g + 1];
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = (j < 16 ? r0 : r1) * f.col[32 * g + j];
        }
        tmem_ld32(tl + 32 * g, s);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = z[j] != 0.f && there ? z[j] * f32(s[j]) : 0.f;
        float run = 0.f;
        tmem_ld32(tl + 128 + 32 * g, s);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          // (rows behind the sequence may hold anything, and a decay of 0 hides a token)
          const float w1 = z[j] != 0.f ? z[j] * f32(s[j]) : 0.f;
          z[j] = g < qw || j <= lane ? run : 0.f;
          run += w1;
        }
        hd.cols[par][qw][32 * g + lane] = column_sums(z);
        if (g < qw) {
          sum += run;
          run = warp_sum(run);
          if (lane == 0) hd.all[par][qw][g] = run;
        }
      }
      hd.rows[par][half][o] = sum;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->bar[GE + par]), mbar_arrive(&ctl->bar[GR]);
      if (!(ok = wait_warp(ctl, GR, it & 1))) break;
      if (half == 0) {  // thread o is token o
        float d = hd.rows[par][0][o] + hd.rows[par][1][o];
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const float u = __shfl_down_sync(0xffffffffu, d, k);
          if (lane + k < 32) d += u;
        }
        for (int r = qw; r < 4; ++r) {
          d += hd.cols[par][r][o];
          for (int g = 0; g < qw && r > qw; ++g) d += hd.all[par][r][g];
        }
        if (there) p.inside[(int64_t)i.unit * p.L + i.t0 + o] = p.scale * d;
      }
      ++it;
    }
    if (!ok) ctl->abort = 1;
  }
  tc_fence_before();
  cta_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
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
// Rows that lie apart (axes may repeat), strides below the map's 2^40 bytes.
bool strides_ok(int64_t B, int64_t H, int64_t L, int d, const Strides& s) {
  auto axis = [&](int64_t n, int64_t st, bool repeats) { return n <= 1 || (repeats && st == 0) || (st >= d && st < 1ll << 38); };
  return axis(B, s.n, true) && axis(H, s.h, true) && axis(L, s.t, false);
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
  const int64_t items = (int64_t)p.B * p.H * chunks, most = ctas_per_wave(2);
  if (items > 0x7f000000ll) return cudaErrorInvalidValue;  // (and a step on top of it)
  return launch_pdl(decay_pairs_kernel<DK, DV>, dim3((unsigned)(items < most ? items : most)), dim3(kPairThreads), Sm::kBytes, s,
                    m, p, chunks, (int)items);
}

}  // namespace

bool decay_tc_rows_ok(int B, int H, int L, int d, const Strides& s) { return strides_ok(B, H, L, d, s); }

// One CTA an SM (152); a state pass takes about 0.6 of the pass's time a chunk.
static int tc_segments(int64_t ctas, int L) { return decay_segments(ctas, 152, (L + kC - 1) / kC, 0.6, 2.0, 4.0); }

size_t decay_tc_workspace(int B, int H, int L, int da, int dc) {
  const int64_t ctas = (int64_t)B * H * (dc / kN);
  return decay_seg_bytes(tc_segments(ctas, L), ctas, da);
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
  DecaySegs& g = q.g;
  g.segs = tc_segments(ctas, a.L);
  g.cps = (chunks + g.segs - 1) / g.segs;
  q.parts = a.fin || a.x ? 3 : 2;
  q.log_scale = log2f(a.scale_in * a.scale_out);
  if (ctas * g.segs > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaError_t e;
  if (g.segs > 1) {
    g.seg_h = ws, g.seg_d = ws + (size_t)g.segs * ctas * a.da * kN;
    TcParams f = q;
    f.g.states_only = true;
    trace_begin("decay_states", s);
    e = a.da == 64 ? launch<64, 1>(m, f, (int)(ctas * (g.segs - 1)), s) : launch<128, 1>(m, f, (int)(ctas * (g.segs - 1)), s);
    trace_end(s);
    ++*launches;
    if (e == cudaSuccess) e = launch_decay_join(a, g, s, launches);
    if (e != cudaSuccess) return e;
  }
  trace_begin("decay_tc", s);
  const int blocks = (int)(ctas * g.segs);
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
  p.inside = a.inside, p.status = a.status;
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
