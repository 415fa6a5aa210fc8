// k_cache_attn.cu -- attention over the 8-bit paged cache for one to a few new tokens per
// sequence (decode, verification of drafts), merged with another branch.
//
// For each (sequence n, key head) the rows are its G = H / Hk query heads times the new
// tokens.  With z the logits in units of log 2, softmax is one pass over the cache:
//   m' = max(m, z),  l' = l 2^(m-m') + sum 2^(z-m'),  o' = o 2^(m-m') + sum 2^(z-m') v.
// The value scales are powers of two 2^e per page, so the weights the tensor cores see are
// 2^(z+e-mo), whatever the pages' scales, with a reference mo of their own, kLift below the
// maximum of z + e when it is set: binary16 holds 2^-24 to 2^16, and what many light tokens next to
// a heavy one weigh is lost at the low end.  m moves with every unit, mo (and with it the
// rescaling of o) only when the maximum has grown by more than kLazy.
//
// What bounds it: the cache is read once, 2 D bytes per token and head, and everything else
// is small; the floor is those bytes at the measured copy rate.  So the work is cut evenly
// over the bytes, not over the sequences: all 32-token units of all (sequence, head) pairs
// form one list, every CTA takes an equal contiguous share of it, and pairs that end up in
// several CTAs are joined by the last of them to finish (fixed order: results do not depend
// on timing).  Inside a CTA every warp owns units of its own, with no CTA-wide barrier in
// the loop: one lane copies the keys, then the values of the next unit with bulk copies
// (pages are contiguous and stored in the order the reads want) while the warp computes.
// The products run on mma.sync: 16 rows fill its M, where the 128 rows of a tcgen05 tile
// would be an eighth full, and the tensor time is a third of the copy time.
//
// Measured, H = 32, Hk = 8, D = 128, one new token, e4m3 (share of the measured copy rate):
//   64 sequences of 8192 tokens 183 us (86%), of 128 to 8192 106 us (75%), in fp32 135 us; one
//   of 131072 tokens 56 us (70%), in fp32 65; 64 x 32 heads, windows of 1024, bytes 117 us (67%),
//   e4m3 101; one sequence of 500 tokens 12 us.  Many rows in fp32 (T = 512, two sequences at 3000:
//   506 us; T = 2048 at 14336: 8.0 ms, 130 TFLOP/s) are bound by their two-part products.
// The loop runs at 6.7 TB/s; the rest is the start (positions, pages, first copies: about 6 us)
// and the end of the slowest warp and the joins after it (10 to 20 us).
#include <algorithm>

#include "kv_cache.cuh"
#include "tc_sm100.cuh"

namespace lz {
namespace {

using tc::mbar_try_wait;

constexpr int kThreads = 256;
constexpr int kUnit = 32;   // tokens per unit of work
constexpr int kBatch = 16;  // units whose pages and scales are looked up at a time
constexpr int kMaxM = 16;
constexpr int kMaxCtas = 304;  // CTAs of a launch at most (sizes the scratch): two per SM
static_assert(kMaxCtas * 8 <= kCacheCounters, "a counter per team");
// From this many (sequence, head) pairs on, each warp works alone: starting and ending a
// segment then stalls one warp of sixteen instead of a CTA's eight (512 pairs, 128 to 8192
// tokens: 132 us against 160).  Below, a pair would be spread over so many warps that joining
// their results costs more (128 pairs, 4096 tokens: 45 us against 39).
constexpr int64_t kSoloSegments = 256;
constexpr float kFar = 60.f;  // see where it is used
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What rounding (lo, hi) to halves lost, again as halves.
__device__ __forceinline__ uint32_t half2_rest(float lo, float hi, uint32_t r) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
  return half2_bits(lo - f.x, hi - f.y);
}

// What the rows of one (sequence, block of rows) see.  `m` counts them: sequence m / RB,
// rows RR * (m % RB) and on (row = token * G + head in group).
struct Segment {
  int64_t base;  // first unit's first token (a multiple of kUnit)
  int64_t p0;    // position of token 0
  int64_t first; // first visible token, >= 0
  int lo, hi;    // visible tokens of the block relative to base; hi < lo: none
  int units;     // >= 1
  int cnt;       // tokens with a query
};

__device__ __forceinline__ Segment segment_of(const CacheAttn& a, int m, int RB, int RR, int G) {
  const int n = m / RB, r0 = (m - n * RB) * RR;
  Segment s;
  s.p0 = a.pos[n];
  s.cnt = a.count ? a.count[n] : a.T;
  s.first = a.first ? max((int64_t)0, a.first[n]) : 0;
  // rows of an unknown count are 0; with a bad position they see no cached token
  const bool known = s.cnt >= 0 && s.cnt <= a.T, placed = position_ok(s.p0);
  if (!known || !placed) raise_status(a.status, kDevCheck);
  s.cnt = known ? s.cnt : 0, s.p0 = placed ? s.p0 : 0;
  s.base = 0, s.lo = 0, s.hi = -1, s.units = 1;
  if (placed && r0 < s.cnt * G) {
    // what the whole sequence sees has to fit its table
    const int64_t all_lo = max(s.first, a.W > 0 ? s.p0 - a.W + 1 : (int64_t)0), all_hi = s.p0 + s.cnt - 1;
    if (all_lo <= all_hi) {
      if (!span_ok(a.c, all_lo, all_hi)) {
        raise_status(a.status, kDevCheck);
      } else {
        const int t0 = r0 / G, t1 = (min(r0 + RR, s.cnt * G) - 1) / G;
        const int64_t lo = max(s.first, a.W > 0 ? s.p0 + t0 - a.W + 1 : (int64_t)0), hi = s.p0 + t1;
        if (lo <= hi) {
          s.base = lo & ~(int64_t)(kUnit - 1);
          s.lo = (int)(lo - s.base);
          s.hi = (int)(hi - s.base);
          s.units = s.hi / kUnit + 1;
        }
      }
    }
  }
  return s;
}

// What a CTA works on between two merges: units ua .. ub-1 of one segment and key head.  Kept
// in shared memory, with the position in the list: none of it is worth a register in the loop.
struct Piece {
  Segment s;
  int64_t f, seg0;      // list indices: of the next piece, of segment m's first entry (head 0)
  int m, n, r0, hk, ua, ub, rows;
  int c0, c1;           // the teams that share the segment and head
  int all_lo, all_hi;   // tokens that every row sees, relative to the segment's base
};

// Where a unit's two 16-token blocks are (in blocks of 16 rows from the pool's start) and, one
// byte each, the exponent bits of their key scales and of their value scales; a key scale of
// 0 (no valid scale is) marks a block with nothing to see.
struct UnitMeta {
  int at0, at1;
  uint32_t exps;  // key 0, key 1, value 0, value 1
};

// Adds 1 to a counter and returns what it was: the writes of this thread's team, ordered before
// by its barrier, become visible with it, and those of the teams that counted before are seen.
__device__ __forceinline__ unsigned count_up(unsigned* p) {
  unsigned v;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// One merged set of rows: maxima, sum and output of a row (unnormalised).
struct RowStat {
  float m, mo, l;
};

// Solo: every warp works through a share of its own, without the others of its CTA.
template <typename T, int D, int F, int RG, bool Solo>
struct Shape {
  static_assert(!Solo || RG == 1, "a warp has 16 rows");
  static constexpr int NS = sizeof(T) == 4 ? 2 : 1;  // parts of a query and of a probability
  static constexpr int TG = Solo ? 1 : 8 / RG;       // groups that share out a piece's units
  static constexpr int NG = 8 / RG;                  // groups of a CTA
  static constexpr int S = RG;                       // stages per unit group
  static constexpr int RR = 16 * RG;                 // rows of a team
  static constexpr int NT = Solo ? 8 : 1;            // teams of a CTA
  static constexpr int kHalf = kUnit * D;            // bytes of the keys of a unit
  // dynamic shared memory: the unit buffers, which the merge of the warps' outputs reuses
  // (8 warps x 16 rows x D floats, the same size), then the queries
  static constexpr int kBuf = NG * S * 2 * kHalf;
  static_assert(kBuf == 8 * 16 * D * 4, "the merge fills the unit buffers");
  static constexpr int kSmem = kBuf + NT * RR * D * 2 * NS;
  // two CTAs per SM where their shared memory allows it
  static constexpr int kPerSm =
      kSmem + NT * RR * (kMaxM + 1) * 4 + NG * 2 * kBatch * (int)sizeof(UnitMeta) + 2560 <= 113 * 1024 ? 2 : 1;
  // Starting a segment costs a team about as much as this many units: the list of work holds
  // that many empty entries in front of every segment, so that teams with many short segments
  // get fewer units.  (3 and 12 instead: 64 uneven sequences 106 -> 110 us, 16 of them 62 -> 66.)
  static constexpr int kSegCost = Solo ? 8 : 20;
  static constexpr int kMinUnits = 4 * TG;  // of a piece, where a segment has them
  // Weights reach 2^(kLift + kLazy), a quarter of binary16's range: logits may be off by their own
  // rounding.  Two parts of a weight resolve 2^-25 / 2^kLift of the largest; fp32 calls, whose
  // rescaling is little beside their products, take most of the range for that.
  static constexpr float kLift = NS == 2 ? 12.f : 6.f, kLazy = 14.f - kLift;
};

template <typename T, int D, int F, int RG, bool Solo>
__global__ void __launch_bounds__(kThreads, Shape<T, D, F, RG, Solo>::kPerSm)
    split_kernel(CacheAttn a, int RB, int prow) {
  using Sh = Shape<T, D, F, RG, Solo>;
  constexpr int NS = Sh::NS, TG = Sh::TG, S = Sh::S, RR = Sh::RR, KS = D / 16, NT = D / 8, NG = Sh::NG;
  constexpr int kSegCost = Sh::kSegCost, kTeams = Sh::NT, kTeam = Solo ? 32 : kThreads;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t s_bar[4][NG * S];  // keys full, values full, keys free, values free
  __shared__ float s_rs_all[kTeams][RR];              // log2 e * scale * the query's power of two
  __shared__ float s_zm_all[kTeams][RR * kMaxM];      // logits of the meta tokens
  __shared__ RowStat s_st[8][16];
  __shared__ UnitMeta s_meta[NG][2][kBatch];  // of each group, two batches
  __shared__ int64_t s_sum[8];
  __shared__ int s_most[8];
  __shared__ Piece s_pieces[kTeams];
  __shared__ int s_abort, s_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int rg = warp % RG, group = warp / RG, tg = Solo ? 0 : group;
  // the team (the CTA, or this warp): its threads, its memory, its barrier
  const int team = Solo ? warp : 0, tt_id = Solo ? lane : tid;
  unsigned char* s_q = smem + Sh::kBuf + (size_t)team * RR * D * 2 * NS;
  float *s_rs = s_rs_all[team], *s_zm = s_zm_all[team];
  Piece& s_p = s_pieces[team];
  auto team_sync = [] {
    if (Solo) __syncwarp();
    else __syncthreads();
  };
  const int G = a.H / a.c.Hk, Hk = a.c.Hk;

  if (tid == 0) {
    for (int i = 0; i < NG * S; ++i) {
      tc::mbar_init(&s_bar[0][i], 1);
      tc::mbar_init(&s_bar[1][i], 1);
      tc::mbar_init(&s_bar[2][i], RG);
      tc::mbar_init(&s_bar[3][i], RG);
    }
    s_abort = 0;
    tc::fence_mbar_init();
  }
  pdl_wait();

  // How the units are shared out.  Either every segment is cut into ceil(units / U) equal pieces,
  // U such that the pieces are at most as many as the teams; or the list of all units
  // (sequence-major, then head, then token, kSegCost empty entries in front of each segment) is
  // cut into equal shares, whatever segments they cross.  A team then has one piece, or often
  // two with a start and a join more: pieces are taken while the longest is not longer than a
  // share by more than half of that cost.  (64 x 32 heads, windows of 1024: 127 us in shares, 116 in
  // pieces; 96 segments of drafted tokens 33 and 27.)
  const int M2 = a.c.N * RB, segs = M2 * Hk;
  const int workers = gridDim.x * kTeams, worker = blockIdx.x * kTeams + team;
  bool pieces = false;
  int64_t U = 1, share = 1, f1, total;
  {
    const int mine = tid < M2 ? segment_of(a, tid, RB, RR, G).units : 0;
    int64_t c = mine;
    int most = mine;
    for (int m = tid + kThreads; m < M2; m += kThreads) {
      const int u = segment_of(a, m, RB, RR, G).units;
      c += u, most = max(most, u);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s_sum[warp] = c, s_most[warp] = most;
    if (tid < kTeams) s_pieces[tid].m = -1;
    __syncthreads();
    int64_t units = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) units += s_sum[w], most = max(most, s_most[w]);
    units *= Hk;
    total = units + (int64_t)segs * kSegCost;
    share = max((total + workers - 1) / workers, (int64_t)(Sh::kMinUnits + kSegCost));
    if ((int64_t)segs * 8 <= workers) {  // the pieces' rounding hardly counts
      U = max((units + workers - segs - 1) / (workers - segs), (int64_t)Sh::kMinUnits);
      pieces = true;
    } else if (segs <= workers) {
      // pieces of U: at most units / U + segs of them, or segs where U is the longest segment
      U = segs < workers ? min((units + workers - segs - 1) / (workers - segs), (int64_t)most) : most;
      U = max(U, (int64_t)Sh::kMinUnits);
      int longest = 0;
      for (int m = tid; m < M2; m += kThreads) {
        const int u = m == tid ? mine : segment_of(a, m, RB, RR, G).units;
        const int k = (int)((u + U - 1) / U);
        longest = max(longest, (u + k - 1) / k);
      }
      longest = __reduce_max_sync(0xffffffffu, longest);
      __syncthreads();
      if (lane == 0) s_most[warp] = longest;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) longest = max(longest, s_most[w]);
      pieces = longest <= share + kSegCost / 2;
    }
    if (pieces) share = 1;
    const int64_t cta_f = (int64_t)blockIdx.x * kTeams * share;  // where the first team starts
    int64_t before = 0;
    for (int m0 = 0; m0 < M2; m0 += kThreads) {
      const int m = m0 + tid;
      int64_t u = 0;
      if (m < M2) {
        const int n_u = m0 == 0 ? mine : segment_of(a, m, RB, RR, G).units;
        u = (pieces ? (n_u + U - 1) / U : (int64_t)n_u + kSegCost) * Hk;
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
      for (int w = 0; w < kTeams; ++w) {
        const int64_t f = cta_f + w * share;
        if (f < c && f >= c - u) s_pieces[w].m = m, s_pieces[w].seg0 = c - u, s_pieces[w].f = f;
      }
      for (int w = 0; w < 8; ++w) before += s_sum[w];
      if (cta_f + (kTeams - 1) * share < before) break;
    }
    __syncthreads();
    f1 = (worker + 1) * share;
    if (!pieces) f1 = min(f1, total);
  }
  uint32_t used = 0;  // units this warp's group has consumed, over all pieces
  auto wait_lane = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long c0 = clock64();
    while (true) {
#pragma unroll 1
      for (int k = 0; k < 32; ++k)
        if (mbar_try_wait(bar, parity)) return true;
      if (*(volatile int*)&s_abort) return false;
      if (clock64() - c0 > 2000000000ll) {
        *(volatile int*)&s_abort = 1;
        return false;
      }
    }
  };
  // one answer for the warp: what follows a wait is executed by all its lanes together
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = wait_lane(bar, parity);
    return __all_sync(0xffffffffu, ok) != 0;
  };

  while (true) {
    if (tt_id == 0) {
      Piece& p = s_p;
      p.ub = 0;
      if (p.m >= 0 && p.f < f1) {
        p.s = segment_of(a, p.m, RB, RR, G);
        p.n = p.m / RB;
        p.r0 = (p.m - p.n * RB) * RR;
        p.rows = max(0, min(RR, p.s.cnt * G - p.r0));
        if (pieces) {
          const int k = (int)((p.s.units + U - 1) / U), i = (int)(p.f - p.seg0);
          p.hk = i / k;
          p.ua = (int)((int64_t)p.s.units * (i - p.hk * k) / k);
          p.ub = (int)((int64_t)p.s.units * (i - p.hk * k + 1) / k);
          p.c0 = (int)p.seg0 + p.hk * k;
          p.c1 = p.c0 + k - 1;
          p.f = f1;
        } else {
          const int entries = p.s.units + kSegCost;
          p.hk = (int)((p.f - p.seg0) / entries);
          const int64_t next = p.seg0 + (int64_t)(p.hk + 1) * entries;
          const int64_t head0 = next - p.s.units;  // this head's first unit
          p.ua = (int)max((int64_t)0, p.f - head0);
          // 0: the share ends before this head's first unit
          p.ub = (int)max((int64_t)0, min((int64_t)p.s.units, f1 - head0));
          p.c0 = (int)(head0 / share);
          p.c1 = (int)((next - 1) / share);
          p.f = next;
        }
        const int64_t last = p.s.p0 + (p.r0 + max(p.rows, 1) - 1) / G;
        p.all_lo = (int)min(max((int64_t)0, max(p.s.first, a.W > 0 ? last - a.W + 1 : (int64_t)0) - p.s.base),
                            (int64_t)0x7fffffff);
        p.all_hi = p.s.hi >= p.s.lo && p.rows > 0 ? (int)(p.s.p0 + p.r0 / G - p.s.base) : -1;
        if (p.hk == Hk - 1) p.seg0 = p.f, ++p.m;
      }
    }
    team_sync();
    if (s_p.ub == 0) break;
    // s_p is read again wherever it is needed: its fields are worth no register in the loop
    const int nu = s_p.ub - s_p.ua > tg ? (s_p.ub - s_p.ua - tg + TG - 1) / TG : 0;  // units of this group

    // ---- pages and scales of the group's units, a batch at a time
    auto load_meta = [&](int batch) {
      const int j = batch * kBatch + lane;
      UnitMeta u{0, 0, 0};
      if (lane < kBatch && j < nu) {
        const int tok = (s_p.ua + tg + j * TG) * kUnit, lo = s_p.s.lo, hi = s_p.s.hi;
        const bool in0 = tok + 15 >= lo && tok <= hi, in1 = tok + 31 >= lo && tok + 16 <= hi;
        const uint32_t pg = (uint32_t)((s_p.s.base + tok) >> a.c.log_p);
        const int row = (int)((s_p.s.base + tok) & (a.c.P - 1));
        const bool small = a.c.P == 16;
        int i0 = -1, i1 = -1;
        if (in0 || (in1 && !small)) {
          i0 = pool_page(a.c, s_p.n, pg);
          if (i0 < 0) raise_status(a.status, kDevCheck);
        }
        i1 = i0;
        if (small && in1) {
          i1 = pool_page(a.c, s_p.n, pg + 1);
          if (i1 < 0) raise_status(a.status, kDevCheck);
        }
        if (in0 && i0 >= 0) {
          const size_t ph = (size_t)i0 * Hk + s_p.hk;
          u.at0 = (int)((ph * a.c.P + row) >> 4);
          u.exps |= (__float_as_uint(a.c.ks[ph]) >> 23 & 0xff) | (__float_as_uint(a.c.vs[ph]) >> 23 & 0xff) << 16;
        }
        if (in1 && i1 >= 0) {
          const size_t ph = (size_t)i1 * Hk + s_p.hk;
          u.at1 = (int)((ph * a.c.P + ((row + 16) & (a.c.P - 1))) >> 4);
          u.exps |= (__float_as_uint(a.c.ks[ph]) >> 23 & 0xff) << 8 | (__float_as_uint(a.c.vs[ph]) >> 23 & 0xff) << 24;
        }
      }
      if (lane < kBatch) s_meta[group][batch & 1][lane] = u;
      __syncwarp();
    };
    // Copies the keys (x = 0) or values (x = 1) of the group's unit j into its stage.
    auto copy = [&](int x, int j) {
      if (lane == 0) {
        const UnitMeta& u = s_meta[group][(j / kBatch) & 1][j % kBatch];
        const int st = group * S + (used + j) % S;
        const bool in0 = u.exps & 0xff, in1 = u.exps & 0xff00;
        unsigned char* dst = smem + (size_t)st * 2 * Sh::kHalf + x * Sh::kHalf;
        const unsigned char* pool = x ? a.c.v : a.c.k;
        uint64_t* bar = &s_bar[x][st];
        constexpr uint32_t half = Sh::kHalf / 2;
        tc::mbar_arrive_expect_tx(bar, half * ((in0 ? 1 : 0) + (in1 ? 1 : 0)));
        if (in0 && in1 && u.at1 == u.at0 + 1) {
          tc::bulk_load(dst, pool + (size_t)u.at0 * half, 2 * half, bar);
        } else {
          if (in0) tc::bulk_load(dst, pool + (size_t)u.at0 * half, half, bar);
          if (in1) tc::bulk_load(dst + half, pool + (size_t)u.at1 * half, half, bar);
        }
      }
      __syncwarp();
    };
    if (rg == 0) {
      load_meta(0);
      for (int j = 0; j < S && j < nu; ++j) copy(0, j), copy(1, j);
    }

    // ---- queries: rotated, scaled to a power of two near 2^13, in the order the MMAs read
    constexpr int LPR = D / 4, RPI = 32 / LPR;  // lanes per row, rows per iteration of a warp
    constexpr int WARPS = Solo ? 1 : 8;
    for (int i = tt_id; i < RR * D * NS / 8; i += kTeam) reinterpret_cast<uint4*>(s_q)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tt_id; i < RR; i += kTeam) s_rs[i] = 0.f;
    team_sync();
    const int d0q = (lane % LPR) * 4;
    for (int rb = (Solo ? 0 : warp) * RPI; rb < s_p.rows; rb += 4 * WARPS * RPI) {
      float x[4][4], y[4][4];
      bool have[4];
      {
        // four rows at a time, dead ones reading the last live one: no branch keeps the loads
        // from being in flight together
        Raw4<T> xr[4], yr[4];
        const T* qp[4];
        const bool half = a.rope.turns && a.rope.layout == LIZARD_ROPE_HALF && d0q < a.rope.rot;
        const int hr = a.rope.rot / 2;
        const int other = half && hr % 4 == 0 ? (d0q < hr ? d0q + hr : d0q - hr) : d0q;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = rb + k * WARPS * RPI + lane / LPR, rr = s_p.r0 + min(r, s_p.rows - 1);
          const int tt = rr / G, h = s_p.hk * G + rr - tt * G;
          have[k] = r < s_p.rows;
          qp[k] = static_cast<const T*>(a.q) + s_p.n * a.sq.n + h * a.sq.h + tt * a.sq.t;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) xr[k] = raw4(qp[k] + d0q), yr[k] = raw4(qp[k] + other);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 v = xr[k].value();
          float4 o = yr[k].value();
          if (half && hr % 4 != 0) {
            auto at = [&](int e) { return e < a.rope.rot ? ld_f(qp[k] + (e < hr ? e + hr : e - hr)) : 0.f; };
            o = make_float4(at(d0q), at(d0q + 1), at(d0q + 2), at(d0q + 3));
          } else if (!half) {
            o = make_float4(v.y, v.x, v.w, v.z);
          }
          x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
          y[k][0] = o.x, y[k][1] = o.y, y[k][2] = o.z, y[k][3] = o.w;
        }
      }
      if (s_p.ua == 0)  // the piece with the first unit adds the meta tokens
        for (int j = 0; j < a.M; ++j) {
          float z[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int h = s_p.hk * G + (s_p.r0 + rb + k * WARPS * RPI + lane / LPR) % G;
            const float4 v = ld4(static_cast<const T*>(a.mk) + ((size_t)h * a.M + j) * D + d0q);
            z[k] = x[k][0] * v.x + x[k][1] * v.y + x[k][2] * v.z + x[k][3] * v.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) z[k] += __shfl_xor_sync(0xffffffffu, z[k], o);
            if (lane % LPR == 0 && have[k])
              s_zm[(rb + k * WARPS * RPI + lane / LPR) * kMaxM + j] = z[k] * (a.scale * kLog2e);
          }
        }
      float co[4], si[4];
      int angle_of = -1;  // token whose angles co, si hold: the heads of a token share them
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int r = rb + k * WARPS * RPI + lane / LPR;
        if (rb + k * WARPS * RPI >= s_p.rows) break;
        float v[4];
        // the arrays are indexed by constants only
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = k == 0 ? x[0][i] : k == 1 ? x[1][i] : k == 2 ? x[2][i] : x[3][i];
        if (a.rope.turns && r < s_p.rows && d0q < a.rope.rot) {
          const int tt = (s_p.r0 + r) / G, hr = a.rope.rot / 2;
          const bool half = a.rope.layout == LIZARD_ROPE_HALF;
          if (tt != angle_of) {
            angle_of = tt;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = d0q + i;
              co[i] = 1.f, si[i] = 0.f;
              if (e < a.rope.rot) {
                const bool low = half ? e < hr : (e & 1) == 0;
                rope_angle(a.rope.turns[half ? (low ? e : e - hr) : e >> 1], s_p.s.p0 + tt, a.rope.factor, co[i], si[i]);
                if (low) si[i] = -si[i];
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float o = k == 0 ? y[0][i] : k == 1 ? y[1][i] : k == 2 ? y[2][i] : y[3][i];
            v[i] = v[i] * co[i] + o * si[i];
          }
        }
        float mx = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        // v = 2^e v', |v'| < 2^14: halves keep 11 bits down to 2^-28 of the row's largest
        int e = (int)(__float_as_uint(mx) >> 23) - 127 - 13;
        e = max(-126, min(e, 113));
        const float inv = exp2_int(-e);
        if (r < s_p.rows) {
          if (lane % LPR == 0) s_rs[r] = a.scale * kLog2e * exp2_int(e);
          // element d = (D/4) t + 4 s + i of row r feeds lane (r%8) t, step s, register 2 (i/2) + r/8%2
          const int t = d0q / (D / 4), s = (d0q % (D / 4)) / 4;
          uint32_t* dst = reinterpret_cast<uint32_t*>(s_q) +
                          ((size_t)((r >> 4) * NS * KS + s) * 32 + (r & 7) * 4 + t) * 4 + ((r >> 3) & 1);
          const uint32_t w0 = half2_bits(v[0] * inv, v[1] * inv), w1 = half2_bits(v[2] * inv, v[3] * inv);
          dst[0] = w0, dst[2] = w1;
          if (NS == 2) {
            dst[KS * 128] = half2_rest(v[0] * inv, v[1] * inv, w0);
            dst[KS * 128 + 2] = half2_rest(v[2] * inv, v[3] * inv, w1);
          }
        }
      }
    }
    team_sync();

    // ---- this warp's rows g and g + 8
    float o[NT][4], mrow[2] = {-INFINITY, -INFINITY}, mo[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    // first token a query at position p sees, relative to the segment's base
    auto sees_from = [&](int64_t p) {
      const int64_t lo = max(s_p.s.first, a.W > 0 ? p - a.W + 1 : (int64_t)0) - s_p.s.base;
      return (int)max((int64_t)0, min(lo, (int64_t)0x7fffffff));
    };
    const bool high = s_p.rows - rg * 16 > 8;
    const uint4* qf = reinterpret_cast<const uint4*>(s_q) + (size_t)rg * NS * KS * 32 + lane;

    for (int j = 0; j < nu; ++j) {
      // the next batch replaces the last one, which no warp of the group (at most S - 1 units
      // behind) still reads half a batch later
      if (rg == 0 && j % kBatch == kBatch / 2 && (j | (kBatch - 1)) + 1 < nu) load_meta(j / kBatch + 1);
      const uint32_t u = used + j;
      const int st = group * S + u % S;
      const uint32_t parity = (u / S) & 1;
      const unsigned char* kb = smem + (size_t)st * 2 * Sh::kHalf;
      const unsigned char* vb = kb + Sh::kHalf;
      const int tok = (s_p.ua + tg + j * TG) * kUnit;
      // logits: lane (g, t4) holds channels (D/4) t4 .. of token 8 i + g
      if (!wait(&s_bar[0][st], parity)) break;
      const UnitMeta& um = s_meta[group][(j / kBatch) & 1][j % kBatch];
      const uint32_t ex = um.exps;
      const bool ok0 = ex & 0xff, ok1 = ex & 0xff00;
      // an unseen block's products become -inf: any positive factor will do
      const float kk[2] = {ok0 ? __uint_as_float((ex & 0xff) << 23) : 1.f,
                           ok1 ? __uint_as_float((ex >> 8 & 0xff) << 23) : 1.f};
      // what makes a logit of row half h's product in block b.  Tiny queries over tiny keys would
      // make it 0, and the -inf of hidden tokens NaN; the smallest normal number makes 0 of any
      // product (below 2^31) just as well.
      auto factor = [&](float r, int b) { return fmaxf(r * kk[b], 0x1p-126f); };
      const float ve[2] = {(float)((int)(ex >> 16 & 0xff) - 127), (float)((int)(ex >> 24) - 127)};
      float z[4][4];
#pragma unroll
      for (int i = 0; i < 4; i += 2) {  // two tiles of 8 tokens share the reads of the queries
        uint32_t w[2][KS];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          z[i + k][0] = z[i + k][1] = z[i + k][2] = z[i + k][3] = 0.f;
          const int r = 8 * (i + k) + g;
#pragma unroll
          for (int h = 0; h < KS / 4; ++h) {
            const uint4 v = *reinterpret_cast<const uint4*>(kb + r * D + 16 * chunk_place<D>(r, KS / 4 * t4 + h));
            w[k][4 * h] = v.x, w[k][4 * h + 1] = v.y, w[k][4 * h + 2] = v.z, w[k][4 * h + 3] = v.w;
          }
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t b[2][2];
          codes_to_half<F>(w[0][s], b[0][0], b[0][1]);
          codes_to_half<F>(w[1][s], b[1][0], b[1][1]);
#pragma unroll
          for (int p = 0; p < NS; ++p) {
            const uint4 q = qf[(p * KS + s) * 32];
            const uint32_t qa[4] = {q.x, q.y, q.z, q.w};
            mma16816(z[i], qa, b[0][0], b[0][1]);
            mma16816(z[i + 1], qa, b[1][0], b[1][1]);
          }
        }
      }
      // the keys' stage is free: the next unit that uses it
      auto refill = [&](int x) {
        // with one warp per group its own reads are done; else the unit before this one,
        // which the other warps have most likely left, is replaced
        const int back = RG > 1 ? 1 : 0;
        if (RG > 1) {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s_bar[2 + x][st]);
        }
        if (rg == 0 && j - back + S < nu && j >= back) {
          if (RG > 1) {
            const uint32_t v = u - 1;
            if (!wait(&s_bar[2 + x][group * S + v % S], (v / S) & 1)) return;
          }
          __syncwarp();
          copy(x, j - back + S);
        }
      };
      refill(0);

      // Row half h (rows g, g + 8) and 16-token block b: z holds raw products, to be multiplied
      // by factor(rs, b).  The upper half is skipped where there are eight rows or fewer.
      const bool whole = ok0 && ok1 && tok >= s_p.all_lo && tok + kUnit - 1 <= s_p.all_hi;
      const float rs[2] = {s_rs[rg * 16 + g], s_rs[rg * 16 + g + 8]};
      if (!whole) {  // column 8 i + 2 t4 + e; at the ends only, so the limits are found here
        int lo_r[2], hi_r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = rg * 16 + g + 8 * i;
          const int64_t p = s_p.s.p0 + (s_p.r0 + r) / G;
          hi_r[i] = s_p.s.hi >= s_p.s.lo && r < s_p.rows ? (int)(p - s_p.s.base) : -1;
          lo_r[i] = sees_from(p);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = tok + 8 * i + 2 * t4 + (e & 1);
            const bool see = (i < 2 ? ok0 : ok1) && c >= lo_r[e >> 1] && c <= hi_r[e >> 1];
            z[i][e] = see ? z[i][e] : -INFINITY;
          }
      }
      float mon[2];
      bool jump = false;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (h == 0 || high) {
          float mn = mrow[h];
          float top = -INFINITY;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float x = fmaxf(fmaxf(z[2 * b][2 * h], z[2 * b][2 * h + 1]),
                            fmaxf(z[2 * b + 1][2 * h], z[2 * b + 1][2 * h + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            x *= factor(rs[h], b);
            mn = fmaxf(mn, x);
            top = fmaxf(top, x + ve[b]);
          }
          mon[h] = fmaxf(mo[h], top - Sh::kLift);
          // the sum's scale follows its maximum exactly, the output's only in steps
          if (mn > mrow[h]) l[h] *= tc::ex2_approx(mrow[h] - mn), mrow[h] = mn;
          jump |= mon[h] > mo[h] + Sh::kLazy;
        }
      if (__any_sync(0xffffffffu, jump)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (h == 0 || high) {
            const float f = mon[h] > mo[h] ? exp2f(mo[h] - mon[h]) : 1.f;
            mo[h] = fmaxf(mo[h], mon[h]);
#pragma unroll
            for (int k = 0; k < NT; ++k) o[k][2 * h] *= f, o[k][2 * h + 1] *= f;
          }
      }
      uint32_t pw[NS][2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 0 || high) {
          const float ml = mrow[h] == -INFINITY ? 0.f : mrow[h], mol = mo[h] == -INFINITY ? 0.f : mo[h];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float f = factor(rs[h], b), sh = mol - ve[b];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x = z[2 * b + i][2 * h], y = z[2 * b + i][2 * h + 1];
              const float p = tc::ex2_approx(fmaf(x, f, -sh)), q = tc::ex2_approx(fmaf(y, f, -sh));
              sum += p + q;
              const uint32_t w = half2_bits(p, q);
              pw[0][b][2 * i + h] = w;
              if (NS == 2) pw[NS - 1][b][2 * i + h] = half2_rest(p, q, w);
            }
            // The weights' sum in units of 2^m.  Where a block's values are so much smaller than
            // the others' that its weights vanish before their share of the sum does, the sum
            // takes exponentials of its own.
            if (__any_sync(0xffffffffu, sh - ml > kFar)) {
              sum = 0.f;
#pragma unroll
              for (int i = 0; i < 2; ++i)
                sum += tc::ex2_approx(fmaf(z[2 * b + i][2 * h], f, -ml)) +
                       tc::ex2_approx(fmaf(z[2 * b + i][2 * h + 1], f, -ml));
              l[h] += sum;
            } else {
              l[h] += sum * tc::ex2_approx(sh - ml);
            }
          }
        } else {
#pragma unroll
          for (int p = 0; p < NS; ++p)
#pragma unroll
            for (int b = 0; b < 2; ++b) pw[p][b][h] = pw[p][b][2 + h] = 0;
        }
      }

      // output: lane (g, t4) holds channels (D/8) g .. of tokens 2 t4, 2 t4 + 1 (+ 8)
      if (!wait(&s_bar[1][st], parity)) break;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        constexpr int WV = D / 32;  // words of a lane's channels
        uint32_t w[4][WV];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 16 * b + 2 * t4 + (k & 1) + 8 * (k >> 1);
          if (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vb + r * D + 16 * chunk_place<D>(r, g));
            w[k][0] = v.x, w[k][1] = v.y, w[k][WV - 2] = v.z, w[k][WV - 1] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(vb + r * D + 16 * chunk_place<D>(r, g >> 1) + 8 * (g & 1));
            w[k][0] = v.x, w[k][1] = v.y;
          }
        }
        if (!whole) {  // what no token was written to may be NaN: 0 times it has to be 0
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = tok + 16 * b + 2 * t4 + (k & 1) + 8 * (k >> 1);
            if (!((b ? ok1 : ok0) && c >= s_p.s.lo && c <= s_p.s.hi)) {
#pragma unroll
              for (int q = 0; q < WV; ++q) w[k][q] = 0;
            }
          }
        }
#pragma unroll
        for (int q = 0; q < WV; ++q) {
          uint32_t b0[4], b1[4];
          codes_to_half<F>(__byte_perm(w[0][q], w[1][q], 0x5140), b0[0], b0[1]);
          codes_to_half<F>(__byte_perm(w[0][q], w[1][q], 0x7362), b0[2], b0[3]);
          codes_to_half<F>(__byte_perm(w[2][q], w[3][q], 0x5140), b1[0], b1[1]);
          codes_to_half<F>(__byte_perm(w[2][q], w[3][q], 0x7362), b1[2], b1[3]);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int p = 0; p < NS; ++p) mma16816(o[4 * q + c], pw[p][b], b0[c], b1[c]);
        }
      }
      refill(1);
    }

    // ---- join the groups' results; then this piece is a partial or the whole
    used += nu;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (t4 == 0) s_st[warp][g + 8 * i] = RowStat{mrow[i], mo[i], l[i]};
    }
    team_sync();  // every unit buffer has been read
    if (*(volatile int*)&s_abort) break;
    float* s_o = reinterpret_cast<float*>(smem);
    constexpr int V4 = D / 4, ROWSTEP = kTeam / V4;
    // o[k][2 i + e] is channel (D/8) (2 t4 + e) + k of row g + 8 i
    const bool whole_seg = s_p.ua == 0 && s_p.ub == s_p.s.units;
    float* part = reinterpret_cast<float*>(a.ws + kCacheParts);
    auto slot = [&](int w, bool starts) { return part + (size_t)(2 * w + (starts ? 1 : 0)) * prow * (D + 4); };
    // Four channels f of row r of warp w: lanes g, t4 write them together, so their places in a
    // row are spread by both.
    auto merge_at = [&](int w, int r, int f) {
      const int t = f / (D / 16);  // the writer's t4
      return reinterpret_cast<float4*>(s_o) + ((size_t)w * 16 + r) * (D / 4) + (f ^ (((r & 7) ^ (t << 1)) & 7));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (rg * 16 + g + 8 * i < s_p.rows)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int k = 0; k < NT; k += 4)
            *merge_at(warp, g + 8 * i, (NT * (2 * t4 + e) + k) / 4) =
                make_float4(o[k][2 * i + e], o[k + 1][2 * i + e], o[k + 2][2 * i + e], o[k + 3][2 * i + e]);
    team_sync();
    auto finish = [&](int r, RowStat s, float4 v, int d0) {
      // row r's 4 channels, normalised and merged
      const int tt = (s_p.r0 + r) / G, h = s_p.hk * G + (s_p.r0 + r) % G;
      const float f = s.l > 0.f ? a.alpha / s.l * exp2f(s.mo - s.m) : 0.f;
      v.x *= f, v.y *= f, v.z *= f, v.w *= f;
      if (a.add) {
        const float4 w = ld4(static_cast<const T*>(a.add) + s_p.n * a.sadd.n + h * a.sadd.h + tt * a.sadd.t + d0);
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
      }
      st4(static_cast<T*>(a.y) + s_p.n * a.sy.n + h * a.sy.h + tt * a.sy.t + d0, v);
    };
    auto join = [](RowStat& s, float4& v, RowStat b, float4 w) {
      const float mm = fmaxf(s.m, b.m), mo2 = fmaxf(s.mo, b.mo);
      const float fa = s.m == mm ? 1.f : exp2f(s.m - mm), fb = b.m == mm ? 1.f : exp2f(b.m - mm);
      const float ga = s.mo == mo2 ? 1.f : exp2f(s.mo - mo2), gb = b.mo == mo2 ? 1.f : exp2f(b.mo - mo2);
      s.l = s.l * fa + b.l * fb;
      v.x = v.x * ga + w.x * gb, v.y = v.y * ga + w.y * gb;
      v.z = v.z * ga + w.z * gb, v.w = v.w * ga + w.w * gb;
      s.m = mm, s.mo = mo2;
    };
    const int d0 = (tt_id % V4) * 4;
    for (int r = tt_id / V4; r < s_p.rows; r += ROWSTEP) {
      RowStat s{-INFINITY, -INFINITY, 0.f};
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < TG; ++q) {
        const int w = Solo ? warp : q * RG + r / 16;
        join(s, v, s_st[w][r % 16], *merge_at(w, r % 16, d0 / 4));
      }
      if (s_p.ua == 0) {
        const int h = s_p.hk * G + (s_p.r0 + r) % G;
        for (int j = 0; j < a.M; ++j) {
          const float z = s_zm[r * kMaxM + j];
          join(s, v, RowStat{z, z, 1.f}, ld4(static_cast<const T*>(a.mv) + ((size_t)h * a.M + j) * D + d0));
        }
      }
      if (whole_seg) {
        finish(r, s, v, d0);
      } else {
        float* p = slot(worker, s_p.ua == 0);
        *reinterpret_cast<float4*>(p + (size_t)r * D + d0) = v;
        if (d0 == 0)
          *reinterpret_cast<float4*>(p + (size_t)prow * D + 4 * r) = make_float4(s.m, s.mo, s.l, 0.f);
      }
    }
    if (s_p.ua == 0)  // queries beyond the sequence's count
      for (int r = s_p.rows + tt_id / V4; r < RR && s_p.r0 + r < a.T * G; r += ROWSTEP) {
        const int tt = (s_p.r0 + r) / G, h = s_p.hk * G + (s_p.r0 + r) % G;
        st4(static_cast<T*>(a.y) + s_p.n * a.sy.n + h * a.sy.h + tt * a.sy.t + d0, make_float4(0.f, 0.f, 0.f, 0.f));
      }
    if (!whole_seg) {
      const int c0 = s_p.c0, c1 = s_p.c1;
      team_sync();
      int last = 0;
      if (tt_id == 0) last = count_up(reinterpret_cast<unsigned*>(a.ws) + c0) == (unsigned)(c1 - c0);
      if (Solo) {
        last = __shfl_sync(0xffffffffu, last, 0);
        __syncwarp();
      } else {
        if (tid == 0) s_last = last;
        __syncthreads();
        last = s_last;
      }
      if (last) {
        // the V4 lanes of a row read the statistics of V4 partials at a time, turn them into
        // weights, and then add the outputs with many loads in flight
        const int k = tt_id % V4;
        constexpr int RW = 4, GROUPS = ROWSTEP;
        int rp = 1;
        while (rp < s_p.rows && rp < GROUPS) rp <<= 1;
        if (!Solo && rp < GROUPS) {
          // fewer rows than groups of lanes: GROUPS / rp groups share out a row's partials
          const int grp = tt_id / V4, r = grp % rp, sub = grp / rp, PS = GROUPS / rp, np = c1 - c0 + 1;
          RowStat s{-INFINITY, -INFINITY, 0.f};
          for (int cb = c0; cb <= c1; cb += V4) {
            float4 b = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
            if (r < s_p.rows && cb + k <= c1)
              b = __ldcg(reinterpret_cast<const float4*>(slot(cb + k, cb + k == c0) + (size_t)prow * D + 4 * r));
            float mm = b.x, mw = b.y;
#pragma unroll
            for (int o = V4 / 2; o > 0; o >>= 1) {
              mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
              mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
            }
            mm = fmaxf(mm, s.m), mw = fmaxf(mw, s.mo);
            float ls = b.x == -INFINITY ? 0.f : b.z * exp2f(b.x - mm);
#pragma unroll
            for (int o = V4 / 2; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
            s = RowStat{mm, mw, (s.m == mm ? s.l : s.l * exp2f(s.m - mm)) + ls};
          }
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          const int ca = c0 + np * sub / PS, cz = c0 + np * (sub + 1) / PS;
          for (int cb = ca; __any_sync(0xffffffffu, cb < cz); cb += V4) {
            float wk = 0.f;
            if (r < s_p.rows && cb + k < cz) {
              const float mo_k = __ldcg(slot(cb + k, cb + k == c0) + (size_t)prow * D + 4 * r + 1);
              if (mo_k != -INFINITY) wk = exp2f(mo_k - s.mo);
            }
            const int cn = min(V4, cz - cb);
            for (int i = 0; __any_sync(0xffffffffu, i < cn); i += 8) {
              float4 x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < s_p.rows && i + e < cn)
                  x[e] = __ldcg(reinterpret_cast<const float4*>(slot(cb + i + e, cb + i + e == c0) + (size_t)r * D + d0));
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float w = __shfl_sync(0xffffffffu, wk, (i + e) & (V4 - 1), V4);
                v.x = fmaf(w, x[e].x, v.x), v.y = fmaf(w, x[e].y, v.y);
                v.z = fmaf(w, x[e].z, v.z), v.w = fmaf(w, x[e].w, v.w);
              }
            }
          }
          float4* s_v = reinterpret_cast<float4*>(s_o);
          s_v[tt_id] = v;
          team_sync();
          if (sub == 0 && r < s_p.rows) {
            for (int q = 1; q < PS; ++q) {
              const float4 w = s_v[(q * rp + r) * V4 + k];
              v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
            }
            finish(r, s, v, d0);
          }
        } else for (int rb = tt_id / V4; rb - tt_id / V4 < s_p.rows; rb += RW * ROWSTEP) {
          RowStat s[RW];
          float4 v[RW];
#pragma unroll
          for (int q = 0; q < RW; ++q) s[q] = RowStat{-INFINITY, -INFINITY, 0.f}, v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int cb = c0; cb <= c1; cb += V4) {
            float wk[RW];
            float4 b[RW];
#pragma unroll
            for (int q = 0; q < RW; ++q) {
              b[q] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
              if (rb + q * ROWSTEP < s_p.rows && cb + k <= c1)
                b[q] = __ldcg(reinterpret_cast<const float4*>(slot(cb + k, cb + k == c0) + (size_t)prow * D +
                                                              4 * (rb + q * ROWSTEP)));
            }
#pragma unroll
            for (int q = 0; q < RW; ++q) {
              float mm = b[q].x, mw = b[q].y;
#pragma unroll
              for (int o = V4 / 2; o > 0; o >>= 1) {
                mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
                mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
              }
              mm = fmaxf(mm, s[q].m), mw = fmaxf(mw, s[q].mo);
              const float fs = s[q].m == mm ? 1.f : exp2f(s[q].m - mm), fv = s[q].mo == mw ? 1.f : exp2f(s[q].mo - mw);
              float ls = b[q].x == -INFINITY ? 0.f : b[q].z * exp2f(b[q].x - mm);
              wk[q] = b[q].y == -INFINITY ? 0.f : exp2f(b[q].y - mw);
#pragma unroll
              for (int o = V4 / 2; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
              s[q] = RowStat{mm, mw, s[q].l * fs + ls};
              v[q].x *= fv, v[q].y *= fv, v[q].z *= fv, v[q].w *= fv;
            }
            const int cn = min(V4, c1 - cb + 1);
            for (int i = 0; i < cn; i += 4) {
              float4 x[RW][4];
#pragma unroll
              for (int q = 0; q < RW; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  x[q][e] = make_float4(0.f, 0.f, 0.f, 0.f);
                  if (rb + q * ROWSTEP < s_p.rows && i + e < cn)
                    x[q][e] = __ldcg(reinterpret_cast<const float4*>(slot(cb + i + e, cb + i + e == c0) +
                                                                     (size_t)(rb + q * ROWSTEP) * D + d0));
                }
#pragma unroll
              for (int q = 0; q < RW; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float w = __shfl_sync(0xffffffffu, wk[q], (i + e) & (V4 - 1), V4);
                  v[q].x = fmaf(w, x[q][e].x, v[q].x), v[q].y = fmaf(w, x[q][e].y, v[q].y);
                  v[q].z = fmaf(w, x[q][e].z, v[q].z), v[q].w = fmaf(w, x[q][e].w, v[q].w);
                }
            }
          }
#pragma unroll
          for (int q = 0; q < RW; ++q)
            if (rb + q * ROWSTEP < s_p.rows) finish(rb + q * ROWSTEP, s[q], v[q], d0);
        }
        if (tt_id == 0) reinterpret_cast<unsigned*>(a.ws)[c0] = 0u;
      }
    }
    // the buffers were written with ordinary stores: order them before the next copies
    tc::fence_proxy_async_smem();
    team_sync();
  }
  if (*(volatile int*)&s_abort) {
    if (tid == 0) raise_status(a.status, kDevTimeout);
    // a wait gave up after a second; copies that other groups issued just before they saw
    // the flag land well within a millisecond
    const long long c0 = clock64();
    while (clock64() - c0 < 4000000ll) {
    }
  }
  pdl_trigger();
}

template <typename T, int D, int F, int RG, bool Solo>
cudaError_t launch_split(const CacheAttn& a, cudaStream_t s, int* launches) {
  using Sh = Shape<T, D, F, RG, Solo>;
  const int rows = a.H / a.c.Hk * a.T, RB = (rows + Sh::RR - 1) / Sh::RR;
  auto* kernel = split_kernel<T, D, F, RG, Solo>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, Sh::kSmem, done);
  if (e != cudaSuccess) return e;
  trace_begin("cache_attn", s);
  e = launch_pdl(kernel, dim3(std::min(ctas_per_wave(Sh::kPerSm), kMaxCtas)), dim3(kThreads), Sh::kSmem, s, a, RB,
                 std::min(rows, Sh::RR));
  trace_end(s);
  ++*launches;
  return e;
}

// Rows of a team, and whether the teams are single warps.
int team_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
bool solo_warps(int N, int Hk, int rows) { return rows <= 16 && (int64_t)N * Hk >= kSoloSegments; }

template <typename T, int D, int F>
cudaError_t by_rows(const CacheAttn& a, cudaStream_t s, int* launches) {
  const int rows = a.H / a.c.Hk * a.T;
  if (solo_warps(a.c.N, a.c.Hk, rows)) return launch_split<T, D, F, 1, true>(a, s, launches);
  switch (team_rows(rows)) {
    case 16: return launch_split<T, D, F, 1, false>(a, s, launches);
    case 32: return launch_split<T, D, F, 2, false>(a, s, launches);
    case 64: return launch_split<T, D, F, 4, false>(a, s, launches);
  }
  // more rows in bf16 run on tcgen05 (cache_attn_tc_used)
  if constexpr (sizeof(T) == 4) return launch_split<T, D, F, 8, false>(a, s, launches);
  return cudaErrorInvalidValue;
}

template <typename T, int D>
cudaError_t by_format(const CacheAttn& a, cudaStream_t s, int* launches) {
  return a.c.fmt == LIZARD_KV_E4M3 ? by_rows<T, D, 0>(a, s, launches) : by_rows<T, D, 1>(a, s, launches);
}

}  // namespace

size_t cache_attn_workspace(int N, int Hk, int H, int T, int d, lizard_dtype dt) {
  if (cache_attn_tc_used(H, Hk, T, dt)) return cache_attn_tc_workspace(d);
  const int rows = H / Hk * T;
  const int teams = kMaxCtas * (solo_warps(N, Hk, rows) ? 8 : 1);
  // the counters, then two partial results per team
  return kCacheParts + (size_t)2 * teams * std::min(rows, team_rows(rows)) * (d + 4) * sizeof(float);
}

cudaError_t launch_cache_attn(const CacheAttn& a, lizard_dtype dt, cudaStream_t s, int* launches) {
  if (cache_attn_tc_used(a.H, a.c.Hk, a.T, dt)) return launch_cache_attn_tc(a, s, launches);
  if (dt == LIZARD_F32)
    return a.c.d == 64 ? by_format<float, 64>(a, s, launches) : by_format<float, 128>(a, s, launches);
  return a.c.d == 64 ? by_format<bf16, 64>(a, s, launches) : by_format<bf16, 128>(a, s, launches);
}

}  // namespace lz
