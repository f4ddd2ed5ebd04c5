// Attention over a paged cache held in 8 bits, with a scale for each block of tokens and
// head, and with a window over the tokens that a row looks back at.
//
//   s_t = scale ks_t q . k8_t,  lse = ln sum_t exp(s_t),  out = sum_t exp(s_t - lse) vs_t v8_t
//
// over the tokens t that the row sees.  The products run on tcgen05 in e4m3, the type the
// cache is held in, straight from the tiles that the copies leave in shared memory:
// nothing is widened.  Tokens are the M dimension: a tile of 128 gives S^T = K Q^T (lanes
// tokens, columns rows) and O^T += V^T P (lanes dims, columns rows, V and P read MN-major).
// So a tile of 8 rows costs an MMA of N = 16, not one padded to 128 rows, a thread has one
// token and with it one K and one V scale, and a row's reference moves with its columns.
//
// What e4m3's four bits lose is kept in a second term, its own columns beside the first:
// q 2^-e = hi + lo / 16 (a bf16 q has eight bits, so this is exact but for what lies
// 2^-21 below the head's largest value), and the weight w = exp(s - ref) vs = hi + lo / 16
// (off by 2^-9 of itself, or by 2^-15 where ref is such that the row's largest w is 32 or
// more: 2^-20 of it).  ref is log2 of a maximum of exp(s) vs seen earlier, less 5; it
// moves (the row's sum and its columns of O rescaled) when a w passes 448, e4m3's largest.
// The sum is of the f32 weights without vs.
//
// A unit of work is (sequence, KV head, R such rows); its tiles are a run of the launch's
// linear list of tiles, of which every CTA (one per SM) takes an equal, contiguous share.
// A unit that lies in one CTA's share is written at once; the parts of any other go to
// the workspace as (O, ref, sum) and a second launch joins them in a fixed order.
//
// The warps: two groups of four do the softmax of every tile, a token per thread and
// half of the rows a group; four copy K and V rows into a ring of slots (16-byte
// cp.async, 128-byte swizzle); one issues S, one P V.
#include "qsa_launch.h"
#include "qsa_share.cuh"
#include "qsa_tc_cache.cuh"

namespace qsa {

namespace {

constexpr int kC8Soft = 8, kC8Prod = 4, kC8MmaS = kC8Soft + kC8Prod, kC8MmaO = kC8MmaS + 1;
constexpr int kC8Warps = 16, kC8Threads = 32 * kC8Warps;  // (the last two only make up a warpgroup)
constexpr int kC8SoftRegs = 160, kC8OtherRegs = 96;  // of 128 a thread at the launch
static_assert(2 * kC8SoftRegs + 2 * kC8OtherRegs <= 4 * 128, "registers of the launch's four warpgroups");
constexpr int kC8T = 128;        // tokens of a tile: the MMAs' M
constexpr int kC8MostRows = 64;  // rows of a unit at most
constexpr int kC8MaxCtas = 160;
constexpr int kC8Start = 4;      // what beginning a unit costs, in tiles
constexpr float kC8Unset = -1e30f;    // a row's reference before it has seen a token
constexpr float kC8Nobody = 1e30f;    // ... of a column without a row: its weights are 0
constexpr float kC8Head = 5.f;        // log2 of a largest w when the reference is set
constexpr float kC8Least = 0x1p-92f;  // a V scale below counts as this for the reference
constexpr long long kC8SpinLimit = 4000000000LL;

template <int HD, int R>
struct C8Geom {
  static constexpr int kN = 2 * R;               // columns: hi terms, lo terms
  static constexpr int kHalves = HD / 128;
  static constexpr uint32_t kQBox = kN * 128, kBox = kC8T * 128, kSlot = kC8T * HD;
  static constexpr int kSlots = HD == 256 ? 5 : 10;
  static constexpr int kS = R < 64 ? 4 : HD == 256 ? 2 : 3;  // S buffers
  static constexpr uint32_t kQBytes = (kHalves * kQBox + 1023) / 1024 * 1024;
  static constexpr uint32_t kPOff = kQBytes, kRingOff = kPOff + 2 * kBox, kCtrlOff = kRingOff + kSlots * kSlot;
  static constexpr uint32_t kSCol = kHalves * kN;  // TMEM: O of each half, then S
  static_assert(kSCol + kS * kN <= 512, "TMEM has 512 columns");
  // kind::f8f6f4, D f32, A and B e4m3, M = 128, N = kN; O: A and B MN-major
  static constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kN >> 3) << 17) | ((128u >> 4) << 24);
  static constexpr uint32_t kIdescO = kIdescS | (1u << 15) | (1u << 16);
};

struct C8Ctrl {
  float factor[kC8MostRows];  // log2 units a unit of S and ks
  float less_ref[kC8MostRows];  // the reference, negated
  float alpha[kC8MostRows], inv[kC8MostRows];
  int32_t depth[kC8MostRows];
  float red[kC8Soft][kC8MostRows / 2];
  uint64_t full[10], empty[10];
  uint64_t s_full[4], s_free[4], p_ready[2], pv_done[4];
  uint64_t q_full, o_free, drain[2];
  int32_t bad[2], abort;
  uint32_t tmem_base;
};
union C8Scratch {  // the plan is made before anything else
  C8Ctrl c;
  ShareScratch share;
};
template <int HD, int R>
constexpr size_t c8_smem() { return C8Geom<HD, R>::kCtrlOff + sizeof(C8Ctrl) + 16; }
static_assert(c8_smem<256, 64>() <= 232448 && c8_smem<128, 64>() <= 232448, "227 KiB per CTA");

struct C8Seq {
  SeqView v;
  int32_t tiles, m_tiles;  // in every unit's list; units of rows, a team's together
  int64_t count;           // tiles of all its units, their starts included
};

// Tiles that hold the first tokens (all of them where there is no window).
__device__ __forceinline__ int32_t first_tiles(const Cache8Args &a, const SeqView &v) {
  return (min(a.n_first, v.ctx + v.rows) + kC8T - 1) / kC8T;
}

// The units' lists have one length: that of the longest where a window cuts them.
template <int R>
__device__ __forceinline__ C8Seq c8_seq(const Cache8Args &a, int team_log, const SeqRaw &raw) {
  C8Seq q;
  q.v = view_seq(a.seqs, raw);
  q.tiles = q.v.rows > 0 ? (q.v.ctx + q.v.rows + kC8T - 1) / kC8T : 0;
  if (a.window > 0 && q.tiles > 0) {
    const int64_t span = (int64_t)a.window + (a.seqs.mask ? q.v.rows : R / a.group + 2);
    q.tiles = (int32_t)min((int64_t)q.tiles, first_tiles(a, q.v) + (span + kC8T - 1) / kC8T + 1);
  }
  q.m_tiles = (int32_t)(((int64_t)q.v.rows * a.group + ((int64_t)R << team_log) - 1) / ((int64_t)R << team_log));
  q.count = q.tiles > 0 ? (int64_t)(q.tiles + kC8Start) * q.m_tiles * a.nkv : 0;
  return q;
}

// One CTA's part of one unit.
struct C8Seg {
  int32_t s, kvh, mt;   // sequence, KV head, this CTA's unit of R rows
  int32_t n;            // tiles to process
  int32_t first, gap;   // tile i of the part is token tile first + i, gap more from `near` on
  int32_t near;
  int32_t back;         // no row sees the tokens from n_first to before `back`
  bool whole, head;     // the unit's every tile; the unit began in an earlier CTA
  bool empty;           // none of its tiles (a share that ends in a unit's start), or no rows
  SeqView v;
  __device__ int32_t tile(int i) const { return first + i + (i >= near ? gap : 0); }
  // whether token t of tile i < n is there and may be seen by a row (others are not read)
  __device__ bool wants(const Cache8Args &a, int32_t t) const { return t < v.ctx + v.rows && (t < a.n_first || t >= back); }
};

// Walks a team's share of the list, unit by unit (each role its own walk), the
// sequences' lengths read one sequence ahead.
template <int R>
struct C8Walk {
  const Cache8Args &a;
  int64_t left, off;
  int32_t s;
  int team_log;
  C8Seq q;
  SeqRaw ahead;
  __device__ C8Walk(const Cache8Args &a_, int team_log_, int32_t s_, int64_t off_, int64_t left_)
      : a(a_), left(left_), off(off_), s(s_), team_log(team_log_) {
    if (left <= 0) return;
    q = c8_seq<R>(a, team_log, read_seq(a.seqs, s));
    ahead = read_seq(a.seqs, min(s + 1, a.seqs.n_seqs - 1));
  }
  __device__ bool next(C8Seg &g) {
    if (left <= 0) return false;
    while (off >= q.count) {
      off -= q.count;
      if (++s >= a.seqs.n_seqs) {
        left = 0;
        return false;
      }
      q = c8_seq<R>(a, team_log, ahead);
      ahead = read_seq(a.seqs, min(s + 1, a.seqs.n_seqs - 1));
    }
    const int32_t length = q.tiles + kC8Start;
    int32_t unit;  // (KV head, team of units of rows)
    if ((off >> 31) == 0) unit = (int32_t)((uint32_t)off / (uint32_t)length);
    else unit = (int32_t)(off / length);
    const int32_t from = (int32_t)(off - (int64_t)unit * length);
    const int32_t part = (int32_t)min((int64_t)(length - from), left);
    off += part;
    left -= part;
    const int32_t i0 = max(0, from - kC8Start), take = max(0, from + part - kC8Start) - i0;
    g.s = s;
    g.kvh = unit / q.m_tiles;
    g.mt = ((unit - g.kvh * q.m_tiles) << team_log) + (int32_t)(blockIdx.x & ((1u << team_log) - 1u));
    g.v = q.v;
    g.whole = take == q.tiles;
    g.head = i0 > 0;
    const int64_t m0 = (int64_t)g.mt * R, m_all = (int64_t)q.v.rows * a.group;
    g.empty = take == 0 || m0 >= m_all;
    g.n = 0;
    if (g.empty) return true;
    // the token tiles that this unit's rows see any of: those of the first tokens, and from
    // `back` (its first row's oldest) to `end` (its last row's newest)
    const bool chain = a.seqs.mask == nullptr;
    const int32_t j0 = (int32_t)(m0 / a.group), j1 = (int32_t)((min(m0 + R, m_all) - 1) / a.group);
    const int32_t end = (q.v.ctx + (chain ? j1 + 1 : q.v.rows) + kC8T - 1) / kC8T;
    g.near = g.gap = g.back = 0;
    if (a.window > 0) {
      g.near = min(end, first_tiles(a, q.v));
      g.back = max(0, q.v.ctx + (chain ? j0 : 0) - (a.window - 1));
      g.gap = max(0, min(g.back / kC8T, end) - g.near);
    }
    g.n = max(0, min(take, end - g.gap - i0));
    g.first = i0;
    g.near = max(0, g.near - i0);
    return true;
  }
};

// Ring position of tile j's V among a part's n tiles, counted from the part's first copy:
// K0, K1, V0, K2, V1, ..., V(n-1), about the order the MMAs take them in.
__device__ __forceinline__ int c8_v_pos(int j, int n) { return j + 1 < n ? 2 + 2 * j : 2 * n - 1; }

__device__ __forceinline__ void mma_e4m3(uint32_t dtmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// This thread's TMEM lane, K consecutive columns; tmem_ready before use.
template <int K>
__device__ __forceinline__ void tmem_cols(uint32_t taddr, uint32_t *v) {
  if constexpr (K == 32) {
    tmem_ld32(taddr, v);
  } else if constexpr (K == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
  } else if constexpr (K == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
  } else {
    static_assert(K == 4, "4, 8, 16 or 32 columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(taddr));
  }
}
// Completes the loads; naming the registers keeps their uses behind it.
template <int K>
__device__ __forceinline__ void tmem_ready(uint32_t *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3])::"memory");
#pragma unroll
  for (int i = 4; i < K; i += 4) asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3])::"memory");
}

__device__ __forceinline__ void tmem_scale1(uint32_t taddr, float by) {
  uint32_t x;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(x)::"memory");
  x = __float_as_uint(__uint_as_float(x) * by);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(x) : "memory");
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A float's place in the order of signed integers, and back.
__device__ __forceinline__ int32_t ordered(float x) {
  const int32_t i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int32_t i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }

// Two values as e4m3 terms hi + lo / 16.  Through f16: its eleven bits hold hi's four and
// the four that lo rounds to (2^-12 of the value is lost beside lo's 2^-9).
__device__ __forceinline__ void split_e4m3(float a, float b, uint32_t &hi, uint32_t &lo) {
  uint32_t w, h;
  uint16_t c, d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(w));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  asm("{\n\t.reg .b32 t, s;\n\tsub.f16x2 t, %1, %2;\n\tmov.b32 s, 0x4C004C00;\n\tmul.f16x2 %0, t, s;\n\t}"  // 16
      : "=r"(w)
      : "r"(w), "r"(h));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(w));
  hi = c;
  lo = d;
}

__device__ __forceinline__ bool any_of_group(int g, bool x) {  // over a softmax group's four warps
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(1 + g)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int g) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + g) : "memory"); }

__device__ __forceinline__ bool nan8(uint32_t byte) { return (byte & 0x7Fu) == 0x7Fu; }

template <int HD, int R>
__global__ void __launch_bounds__(kC8Threads, 1)
cache8_attn_kernel(const Cache8Args a, const FastDiv group_div, int team_log, int64_t *__restrict__ base_out,
                   float2 *__restrict__ part_ml, float *__restrict__ part_o, int32_t *__restrict__ row_seq) {
  using G = C8Geom<HD, R>;
  extern __shared__ __align__(1024) uint8_t c8_shared[];
  C8Scratch &both = *reinterpret_cast<C8Scratch *>(c8_shared + G::kCtrlOff);
  C8Ctrl &C = both.c;
  const uint32_t sQ = sm32(c8_shared), sP = sm32(c8_shared + G::kPOff), sRing = sm32(c8_shared + G::kRingOff);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long lim = a.wait_limit > 0 ? a.wait_limit : kC8SpinLimit;
  volatile int32_t *abort_flag = &C.abort;

  grid_dependency_sync();  // before TMEM too: an earlier launch may hold it
  // ---- the plan (CTA 0 also leaves the sums for the joining launch)
  const uint32_t teams = gridDim.x >> team_log, my_team = blockIdx.x >> team_log;
  const FoundShare found = find_share(a.seqs.n_seqs, kC8Threads, teams, my_team, both.share, [&](int32_t s) -> int64_t {
    if (s >= a.seqs.n_seqs) return 0;
    return c8_seq<R>(a, team_log, read_seq(a.seqs, s)).count;
  });
  if (blockIdx.x == 0) {
    int64_t before = 0;
    for (int32_t s0 = 0; s0 < a.seqs.n_seqs && warp == 0; s0 += 32) {
      const int32_t s = s0 + lane;
      int64_t count = 0;
      if (s < a.seqs.n_seqs) {
        const C8Seq q = c8_seq<R>(a, team_log, read_seq(a.seqs, s));
        if (!q.v.ok) report_error(a.status, kErrRowRange, s);
        count = q.count;
      }
      const int64_t incl = warp_scan(count, lane);
      if (s < a.seqs.n_seqs) base_out[s] = before + incl - count;
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (tid == 0) base_out[a.seqs.n_seqs] = before;
  }
  __syncthreads();  // the plan's scratch lies where the barriers do
  if (tid == 0) {
    for (int i = 0; i < G::kSlots; ++i) {
      mbar_init(sm32(&C.full[i]), 32 * kC8Prod);
      mbar_init(sm32(&C.empty[i]), 1);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(sm32(&C.s_full[b]), 1);
      mbar_init(sm32(&C.s_free[b]), kC8Soft);
      mbar_init(sm32(&C.pv_done[b]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sm32(&C.p_ready[b]), kC8Soft);
      mbar_init(sm32(&C.drain[b]), 1);
      C.bad[b] = 0;
    }
    mbar_init(sm32(&C.q_full), kC8Soft);
    mbar_init(sm32(&C.o_free), kC8Soft);
    C.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kC8MmaS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm32(&C.tmem_base)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem_base;
  const bool laid_out = (sQ & 1023u) == 0;  // the swizzle needs it; the declaration asks for it
  if (warp < kC8Soft) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kC8SoftRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kC8OtherRegs));
  C8Walk<R> walk(a, team_log, found.seq, found.off, laid_out ? found.share.n : 0);
  C8Seg g;

  if (warp >= kC8Soft && warp < kC8MmaS) {
    // ---- producers: warp p brings 32 of a tile's tokens, 512 bytes an instruction (kRows
    // rows); lane i looks up the pool row of its token.  A slot's barrier takes each
    // thread's arrival when its copies have landed, so the whole ring may be in flight.
    constexpr int kCh = HD / 16, kRows = 32 / kCh, kN = 32 / kRows;
    const int p0 = (warp - kC8Soft) * 32, ch = lane % kCh, hl = lane / kCh;
    const uint32_t dst0 = sRing + (uint32_t)(ch >> 3) * G::kBox + (uint32_t)(p0 + hl) * 128u;
    uint32_t ns = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      auto fetch = [&](int j) -> int32_t {  // pool row of this lane's token of tile j, -1: zeros
        if (j >= g.n) return -1;
        const int32_t t = g.tile(j) * kC8T + p0 + lane;
        if (!g.wants(a, t)) return -1;
        const int64_t slot = token_slot(a.seqs, g.s, t);
        if (slot < 0) report_error(a.status, kErrTokenRange, g.s);
        return slot < 0 ? -1 : (int32_t)(slot * a.nkv + g.kvh);
      };
      // Pool rows of this thread's copies of a slot, spread from the lanes that looked them
      // up before the slot is waited for.
      auto spread = [&](int32_t y, int32_t (&r)[kN]) {
#pragma unroll
        for (int k = 0; k < kN; ++k) r[k] = __shfl_sync(0xffffffffu, y, kRows * k + hl);
      };
      auto bring = [&](const uint8_t *pool, const int32_t (&r)[kN]) {
        const uint32_t slot = ns % G::kSlots;
        if (!tc_warp_wait_ready(sm32(&C.empty[slot]), ((ns / G::kSlots) & 1u) ^ 1u, lim, abort_flag)) {
          ok = false;
          return;
        }
        __syncwarp();
        const uint8_t *src = pool + ch * 16;
#pragma unroll
        for (int k = 0; k < kN; ++k)  // row p0 + kRows k + hl, its 16-byte chunks swizzled by row % 8
          cp_async16(dst0 + slot * G::kSlot + (uint32_t)(k * kRows) * 128u + (uint32_t)(((ch & 7) ^ ((kRows * k + hl) & 7)) << 4),
                     src + (int64_t)max(r[k], 0) * HD, r[k] >= 0 ? 16u : 0u);
        cp_async_arrive(sm32(&C.full[slot]));
        ++ns;
      };
      if (g.n > 0) {
        int32_t rv[kN], rk[kN];
        int32_t y = fetch(0);
        spread(y, rv);
        y = fetch(1);
        bring(a.k_pool, rv);
        for (int j = 0; j < g.n && ok; ++j) {
          spread(y, rk);
          y = fetch(j + 2);
          if (j + 1 < g.n) bring(a.k_pool, rk);
          if (ok) bring(a.v_pool, rv);
#pragma unroll
          for (int k = 0; k < kN; ++k) rv[k] = rk[k];
        }
      }
      if (warp == kC8Soft && !g.whole && !g.empty) {  // the rows of a part, for the join
        const int64_t m0 = (int64_t)g.mt * R, m1 = min(m0 + R, (int64_t)g.v.rows * a.group);
        const int32_t end = fast_div(group_div, (int32_t)m1 - 1);
        for (int32_t j = fast_div(group_div, (int32_t)m0) + lane; j <= end; j += 32) row_seq[g.v.row0 + j] = g.s;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives the CTA
  } else if (warp > kC8MmaO) {
    // nothing to do
  } else if (warp >= kC8MmaS) {
    // ---- MMA issuers, one thread each
    if (lane == 0) {
      bool ok = true;
      auto wait = [&](uint64_t &bar, uint32_t parity) {
        ok = ok && tc_wait_ready(sm32(&bar), parity, lim, abort_flag);
        return ok;
      };
      uint32_t slot = 0, phase = 0;  // of the ring
      auto step = [&](uint32_t n) {
        slot += n;
        if (slot >= (uint32_t)G::kSlots) {
          slot -= (uint32_t)G::kSlots;
          phase ^= 1u;
        }
      };
      // The slot holds its copy.  A parity tells two phases apart, so the slot's copy
      // before this one has to be known to have landed.  S of tile j: that one is K, of a
      // tile whose S this thread issued, or V of tile j - 4 or an earlier one, whose P V
      // was waited for, or, in a part's first tiles, V of a part before the last, whose
      // output was written before this part's Q was fetched.  P V of tile j: it is V, or K
      // of an earlier tile.
      auto landed = [&]() {
        if (!wait(C.full[slot], phase)) return false;
        // the copies wrote through the generic proxy; the MMAs read through the async one
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_after();
        return true;
      };
      const uint32_t desc_hi = (uint32_t)(sw128_desc(0) >> 32);
      uint32_t jg = 0, part = 0;  // tiles and parts before this one
      if (warp == kC8MmaS) {
        const uint32_t q_lo = (uint32_t)sw128_desc(sQ), r_lo = (uint32_t)sw128_desc(sRing);
        uint32_t b = 0, b_phase = 1;  // S buffer, parity of its s_free phase before this use
        while (ok && walk.next(g)) {
          if (g.n == 0) continue;
          if (!wait(C.q_full, part & 1u)) break;
          ++part;
          for (int j = 0; j < g.n; ++j, ++jg) {
            if (jg >= (uint32_t)G::kS && !wait(C.s_free[b], b_phase)) break;  // tile j - kS is read
            if (jg >= 4 && !wait(C.pv_done[jg & 3u], ((jg >> 2) & 1u) ^ 1u)) break;
            if (j > 0) step(j == 1 ? 1u : 2u);
            if (!landed()) break;
            const uint32_t d = tmem + G::kSCol + b * G::kN, k_lo = r_lo + slot * (G::kSlot >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk) {
              const uint32_t in = (uint32_t)(kk & 3) * 2u;  // 32 bytes
              mma_e4m3(d, desc_of(k_lo + (uint32_t)(kk >> 2) * (G::kBox >> 4) + in, desc_hi),
                       desc_of(q_lo + (uint32_t)(kk >> 2) * (G::kQBox >> 4) + in, desc_hi), G::kIdescS, kk > 0 ? 1u : 0u);
            }
            mma_commit(sm32(&C.empty[slot]));
            mma_commit(sm32(&C.s_full[b]));
            if (++b == (uint32_t)G::kS) {
              b = 0;
              b_phase ^= 1u;
            }
          }
          step(g.n == 1 ? 2u : 3u);  // past V(n - 2) and V(n - 1)
        }
      } else {
        const uint32_t r_lo = (uint32_t)sw128_mn_desc(sRing, 0), p_lo = (uint32_t)sw128_mn_desc(sP, 0);
        while (ok && walk.next(g)) {
          if (g.n == 0) continue;
          if (part > 0 && !wait(C.o_free, (part - 1) & 1u)) break;  // the part before has left O
          ++part;
          for (int j = 0; j < g.n; ++j, ++jg) {
            if (!wait(C.p_ready[jg & 1u], (jg >> 1) & 1u)) break;
            step(j + 1 < g.n ? 2u : 1u);
            if (!landed()) break;
            const uint32_t p = p_lo + (jg & 1u) * (G::kBox >> 4), v_lo = r_lo + slot * (G::kSlot >> 4);
#pragma unroll
            for (int h = 0; h < G::kHalves; ++h)
#pragma unroll
              for (int kk = 0; kk < kC8T / 32; ++kk)  // 32 tokens a step: 4 KiB of V's and of P's rows
                mma_e4m3(tmem + (uint32_t)h * G::kN, desc_of(v_lo + (uint32_t)h * (G::kBox >> 4) + 256u * kk, desc_hi),
                         desc_of(p + 256u * kk, desc_hi), G::kIdescO, (j > 0 || kk > 0) ? 1u : 0u);
            mma_commit(sm32(&C.empty[slot]));
            mma_commit(sm32(&C.pv_done[jg & 3u]));
          }
          step(1u);
        }
      }
      // every MMA this thread issued has finished before TMEM is freed
      mma_commit(sm32(&C.drain[warp - kC8MmaS]));
      tc_wait(sm32(&C.drain[warp - kC8MmaS]), 0u, kC8SpinLimit, nullptr);
    }
    __syncwarp();
  } else {
    // ---- softmax: group w has rows [w R/2, w R/2 + R/2) of every tile, thread tk the
    // tile's token tk (TMEM lane) and, at the end, dims tk and tk + 128.  After an abort
    // every wait returns at once, and the loops and barriers run on to the end.
    constexpr int kHalf = R / 2, kAtOnce = kHalf < 16 ? kHalf : 16;  // its rows, rows of a TMEM load
    const int w = warp >> 2, wq = warp & 3, tk = wq * 32 + lane, n0 = w * kHalf;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    auto wait_pv = [&](uint32_t i) { tc_warp_wait_ready(sm32(&C.pv_done[i & 3u]), (i >> 2) & 1u, lim, abort_flag); };
    // This warp's rows of a part's Q, split into two e4m3 terms, with what goes with a row.
    auto load_q = [&](const C8Seg &e) {
      const int64_t m0 = (int64_t)e.mt * R, m_all = (int64_t)e.v.rows * a.group;
      constexpr int kLanes = HD / 8, kPer = 32 / kLanes;  // lanes a row, rows a warp takes at once
      const int ch = lane % kLanes, sub = lane / kLanes;
#pragma unroll 1
      for (int i = wq * kPer; i < kHalf; i += 4 * kPer) {
        const int n = n0 + i + sub;
        const bool mine = i + sub < kHalf, valid = mine && m0 + n < m_all;
        const int32_t m = valid ? (int32_t)(m0 + n) : 0, j = fast_div(group_div, m);
        const int32_t head = e.kvh * a.group + (m - j * a.group);
        float x[8], amax = 0.f;
        unpack8(valid ? ldg_v4(a.q + (int64_t)(e.v.row0 + j) * a.q_stride + (int64_t)head * HD + 8 * ch) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(x[k]) < INFINITY ? fabsf(x[k]) : 0.f);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // the least power of two s with amax <= 448 s = 1.75 * 2^8 s, and 1 / s
        const uint32_t u = __float_as_uint(amax);
        const int ex = max(-126, (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0));
        const float s = __uint_as_float((uint32_t)(127 + ex) << 23), inv = __uint_as_float((uint32_t)(127 - ex) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)  // (x + 0 x: an infinity becomes NaN, which the conversions keep)
          split_e4m3(fmaf(x[2 * k], 0.f, x[2 * k]) * inv, fmaf(x[2 * k + 1], 0.f, x[2 * k + 1]) * inv, hi[k], lo[k]);
        if (mine) {
          auto at = [&](int row) {  // 8 bytes of a 128-byte row of a box, its 16-byte chunks swizzled
            const int byte = 8 * ch;
            return c8_shared + (byte >> 7) * G::kQBox + row * 128 + (((byte >> 4) & 7) ^ (row & 7)) * 16 + (byte & 8);
          };
          *reinterpret_cast<uint2 *>(at(n)) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2 *>(at(R + n)) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        }
        int32_t depth = 0;
        if (a.window > 0 && a.seqs.mask != nullptr && valid) {  // the row's drafted tokens, over its lanes
          const uint32_t *mrow = a.seqs.mask + (int64_t)(e.v.row0 + j) * a.seqs.mask_words;
          for (int32_t k = ch; 32 * k < e.v.rows; k += kLanes) {
            const int32_t over = e.v.rows - 32 * k;
            depth += __popc(over >= 32 ? mrow[k] : mrow[k] & ((1u << over) - 1u));
          }
        }
        if (a.window > 0 && a.seqs.mask != nullptr) {
#pragma unroll
          for (int o = kLanes / 2; o; o >>= 1) depth += __shfl_xor_sync(0xffffffffu, depth, o);
        }
        if (mine && ch == 0) {
          C.factor[n] = a.scale_log2 * s;
          C.less_ref[n] = valid ? -kC8Unset : -kC8Nobody;
          C.depth[n] = max(0, depth - 1);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(sm32(&C.q_full));
    };
    uint32_t jg = 0, ns = 0;
    int32_t seg = 0;
    bool more = walk.next(g);
    if (more && g.n > 0) load_q(g);
    while (more) {
      ++seg;
      const int64_t m0 = (int64_t)g.mt * R, m_all = (int64_t)g.v.rows * a.group;
      const int32_t kv = g.v.ctx + g.v.rows;
      const bool chain = a.seqs.mask == nullptr;
      // whether a row may be blind to a token that another one sees, or that is read beside its own
      const bool veiled = g.v.rows > 1 || !chain || a.window > 0;
      const int32_t j0 = g.empty ? 0 : fast_div(group_div, (int32_t)m0);
      const int32_t j1 = g.empty ? 0 : fast_div(group_div, (int32_t)(min(m0 + R, m_all) - 1));
      // tokens below `clear` and, of a window, from `old` on or below n_first are seen by every row
      const int32_t clear = chain ? g.v.ctx + j0 + 1 : g.v.ctx;
      const int32_t old = a.window > 0 ? g.v.ctx + (chain ? j1 : g.v.rows - 1) - (a.window - 1) : 0;
      auto is_masked = [&](int32_t t0) { return t0 + kC8T > clear || (t0 < old && t0 + kC8T > a.n_first); };
      // whether row n sees token t
      auto sees = [&](int n, int32_t t) -> bool {
        if (m0 + n >= m_all || t >= kv) return false;
        const int32_t j = fast_div(group_div, (int32_t)(m0 + n));
        const bool drafted = t >= g.v.ctx;
        if (!chain && drafted)
          return sees_draft(a.seqs.mask + (int64_t)(g.v.row0 + j) * a.seqs.mask_words, j, t - g.v.ctx);
        const int32_t at = g.v.ctx + (chain ? j : C.depth[n]);
        return t <= at && (a.window == 0 || t < a.n_first || at - t < a.window);
      };
      // K and V scales of this thread's token: their block two tiles ahead, they one
      auto block_of = [&](int j) -> int32_t {
        if (j >= g.n) return -1;
        const int32_t t = g.tile(j) * kC8T + tk;
        if (!g.wants(a, t)) return -1;
        const int64_t slot = token_slot(a.seqs, g.s, t);
        return slot < 0 ? -1 : (int32_t)((slot >> a.unit_log) * a.nkv) + g.kvh;
      };
      float ks = 0.f, vs = 0.f, ks_next = 0.f, vs_next = 0.f;
      int32_t block = block_of(0);
      if (block >= 0) {
        ks_next = a.k_scale[block];
        vs_next = a.v_scale[block];
      }
      block = block_of(1);
      uint64_t sum2[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) sum2[i] = 0ull;
      for (int j = 0; j < g.n; ++j, ++jg) {
        ks = ks_next;
        vs = vs_next;
        ks_next = vs_next = 0.f;
        if (block >= 0) {
          ks_next = a.k_scale[block];
          vs_next = a.v_scale[block];
        }
        block = block_of(j + 2);
        const uint32_t b = jg % (uint32_t)G::kS, sc = lane_base + G::kSCol + b * G::kN + n0;
        const int32_t t0 = g.tile(j) * kC8T;
        const bool masked = is_masked(t0);
        uint32_t see = 0xFFFFFFFFu;
        if (masked) {
          see = 0u;
#pragma unroll 4
          for (int i = 0; i < kHalf; ++i) see |= sees(n0 + i, t0 + tk) ? 1u << i : 0u;
        }
        if (!(ks >= 0.f && ks < INFINITY && vs >= 0.f && vs < INFINITY)) {
          if (see != 0u) report_error(a.status, kErrNonFinite, g.s);
          ks = vs = 0.f;
        }
        const float vx = fmaxf(vs, kC8Least);
        tc_warp_wait_ready(sm32(&C.s_full[b]), (jg / (uint32_t)G::kS) & 1u, lim, abort_flag);
        tc_fence_after();
        float x[kHalf];
        const uint64_t ks2 = pair_f32(ks, ks), sixteenth = pair_f32(0.0625f, 0.0625f);
        // Logits in log2 units, rounded as they are: a reference taken from them is then met
        // exactly, however large they are.
        auto logits = [&]() {
#pragma unroll
          for (int c = 0; c < kHalf; c += kAtOnce) {
            uint32_t hi[kAtOnce], lo[kAtOnce];
            tmem_cols<kAtOnce>(sc + c, hi);
            tmem_cols<kAtOnce>(sc + R + c, lo);
            tmem_ready<kAtOnce>(hi);
            tmem_ready<kAtOnce>(lo);
#pragma unroll
            for (int i = 0; i < kAtOnce; i += 2) {
              const uint64_t s2 = fma2(pair_f32(__uint_as_float(lo[i]), __uint_as_float(lo[i + 1])), sixteenth,
                                       pair_f32(__uint_as_float(hi[i]), __uint_as_float(hi[i + 1])));
              const uint64_t f2 = pair_f32(C.factor[n0 + c + i], C.factor[n0 + c + i + 1]);
              unpair_f32(mul2(mul2(s2, ks2), f2), x[c + i], x[c + i + 1]);
            }
          }
        };
        auto weights = [&]() -> float {  // exp of the logits relative to the references; their largest
          float most = 0.f;
#pragma unroll
          for (int i = 0; i < kHalf; i += 2) {
            float lo, hi;
            unpair_f32(add2(pair_f32(x[i], x[i + 1]), pair_f32(C.less_ref[n0 + i], C.less_ref[n0 + i + 1])), lo, hi);
            x[i] = ex2(lo);
            x[i + 1] = ex2(hi);
            if (masked) {
              if (!((see >> i) & 1u)) x[i] = 0.f;
              if (!((see >> i) & 2u)) x[i + 1] = 0.f;
            }
            most = max3(most, x[i], x[i + 1]);
          }
          return most;
        };
        logits();
        const float most = weights();
        if (any_of_group(w, most * vx > 448.f)) {
          // references move: of the rows whose largest w of this tile is over 2^8
          logits();
          const float lv = log2f(vx);
#pragma unroll
          for (int i = 0; i < kHalf; ++i) {
            const float l = ((see >> i) & 1u) ? x[i] + lv : -INFINITY;
            const float top = unordered(__reduce_max_sync(0xffffffffu, ordered(l != l ? -INFINITY : l)));
            if (lane == i) C.red[warp][i] = top;
          }
          group_sync(w);
          if (tk < kHalf) {
            const float l = fmaxf(fmaxf(C.red[4 * w][tk], C.red[4 * w + 1][tk]), fmaxf(C.red[4 * w + 2][tk], C.red[4 * w + 3][tk]));
            const float was = -C.less_ref[n0 + tk], now = l - kC8Head;
            const bool move = l > was + 8.f;
            C.alpha[n0 + tk] = move ? ex2(was - now) : 1.f;
            if (move) C.less_ref[n0 + tk] = -now;
          }
          group_sync(w);
          if (j > 0) {  // O holds the earlier tiles of this part
            wait_pv(jg - 1);
            tc_fence_after();
          }
#pragma unroll
          for (int i = 0; i < kHalf / 2; ++i) sum2[i] = mul2(sum2[i], pair_f32(C.alpha[n0 + 2 * i], C.alpha[n0 + 2 * i + 1]));
          if (j > 0) {
#pragma unroll 1
            for (int i = 0; i < kHalf; ++i) {
              const float by = C.alpha[n0 + i];
              if (by == 1.f) continue;
#pragma unroll
              for (int h = 0; h < G::kHalves; ++h) {
                tmem_scale1(lane_base + (uint32_t)(h * G::kN + n0 + i), by);
                tmem_scale1(lane_base + (uint32_t)(h * G::kN + R + n0 + i), by);
              }
            }
            tmem_wait_st();
          }
          weights();
        }
        if (jg >= 2) wait_pv(jg - 2);  // P's buffer is free
        // The row of the P buffer that is this token's: the group's bytes of hi and of lo.
        // The sums keep 32 bits, as lse has to; the weights go to the two terms above.
        uint8_t *prow = c8_shared + G::kPOff + (jg & 1u) * G::kBox + tk * 128;
        uint32_t ph[(kHalf + 3) / 4], pl[(kHalf + 3) / 4];
#pragma unroll
        for (int i = 0; i < kHalf; i += 4) {
          uint32_t h[2], l[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint64_t p2 = pair_f32(x[i + 2 * k], x[i + 2 * k + 1]);
            float w0, w1;
            unpair_f32(mul2(p2, pair_f32(vs, vs)), w0, w1);
            split_e4m3(w0, w1, h[k], l[k]);
            sum2[i / 2 + k] = add2(sum2[i / 2 + k], p2);
          }
          ph[i / 4] = h[0] | h[1] << 16;
          pl[i / 4] = l[0] | l[1] << 16;
        }
        auto put = [&](int col, const uint32_t *v) {
          if constexpr (kHalf >= 16) {
#pragma unroll
            for (int c = 0; c < kHalf / 16; ++c)
              *reinterpret_cast<uint4 *>(prow + ((((col >> 4) + c) ^ (tk & 7)) << 4)) =
                  make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
          } else if constexpr (kHalf == 8) {
            *reinterpret_cast<uint2 *>(prow + (((col >> 4) ^ (tk & 7)) << 4) + (col & 8)) = make_uint2(v[0], v[1]);
          } else {
            *reinterpret_cast<uint32_t *>(prow + (((col >> 4) ^ (tk & 7)) << 4) + (col & 12)) = v[0];
          }
        };
        put(n0, ph);
        put(R + n0, pl);
        if (masked && veiled) {
          // A NaN of V would reach, as 0 x NaN, the rows that do not see its token: it is
          // cleared here and given to the rows that do see it when the output is written.
          // (The slot's earlier copy is known to have landed once P V of the tile before the
          // last is done.)
          const uint32_t at = ns + (uint32_t)c8_v_pos(j, g.n), slot = at % G::kSlots;
          tc_warp_wait_ready(sm32(&C.full[slot]), (at / G::kSlots) & 1u, lim, abort_flag);
          __syncwarp();
          uint4 *vt = reinterpret_cast<uint4 *>(c8_shared + G::kRingOff + slot * G::kSlot);
          for (int i = warp * 32 + lane; i < (int)(G::kSlot / 16); i += 32 * kC8Soft) {
            const uint4 x = vt[i];
            uint32_t e[4] = {x.x, x.y, x.z, x.w};
            bool hit = false;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int c = 0; c < 32; c += 8)
                if (nan8(e[k] >> c)) {
                  e[k] &= ~(0xFFu << c);
                  hit = true;
                }
            if (hit) {
              vt[i] = make_uint4(e[0], e[1], e[2], e[3]);
              *reinterpret_cast<volatile int32_t *>(&C.bad[seg & 1]) = seg;
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(sm32(&C.s_free[b]));
          mbar_arrive(sm32(&C.p_ready[jg & 1u]));
        }
      }
      ns += (uint32_t)(2 * g.n);
      C8Seg next;
      const bool more_next = walk.next(next);
      if (!g.empty) {
        // the rows' sums over this group's threads, in a fixed order
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          float even, odd;
          unpair_f32(sum2[i / 2], even, odd);
          float x = i & 1 ? odd : even;
#pragma unroll
          for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (lane == i) C.red[warp][i] = x;
        }
      }
      const int64_t part = (int64_t)blockIdx.x * 2 + (g.head ? 0 : 1);
      group_sync(w);
      if (!g.empty && tk < kHalf) {
        const int n = n0 + tk;
        const float all = (C.red[4 * w][tk] + C.red[4 * w + 1][tk]) + (C.red[4 * w + 2][tk] + C.red[4 * w + 3][tk]);
        const float ref = g.n > 0 ? -C.less_ref[n] : kC8Unset;
        C.inv[n] = all == 0.f ? 0.f : 1.f / all;
        if (m0 + n < m_all) {
          if (!g.whole) {
            part_ml[part * R + n] = make_float2(ref, all);
          } else if (a.lse) {
            const int32_t m = (int32_t)(m0 + n), j = fast_div(group_div, m);
            a.lse[(int64_t)(g.v.row0 + j) * a.nq + g.kvh * a.group + (m - j * a.group)] =
                all == 0.f ? -INFINITY : (ref + log2f(all)) * 0.6931471805599453f;
          }
        }
      }
      bool fix = false;
      if (g.n > 0) {  // S and P V of every tile are done: Q may go, O may be read
        wait_pv(jg - 1);
        tc_fence_after();
        __syncwarp();
        fix = *reinterpret_cast<volatile int32_t *>(&C.bad[seg & 1]) == seg;
      }
      if (fix) {  // rare: rows that see a cleared NaN; the rows' depths are still this part's
        for (int i = 0; i < kHalf; ++i) {
          for (int h = 0; h < G::kHalves; ++h) {
            bool hit = false;
            for (int j = 0; j < g.n; ++j) {
              const int32_t t0 = g.tile(j) * kC8T;
              if (!is_masked(t0)) continue;
              for (int32_t t = t0; t < min(kv, t0 + kC8T); ++t) {
                if (!sees(n0 + i, t)) continue;
                const int64_t slot = token_slot(a.seqs, g.s, t);
                hit = hit || (slot >= 0 && nan8(a.v_pool[(slot * a.nkv + g.kvh) * HD + h * 128 + tk]));
              }
            }
            uint32_t x;
            __syncwarp();
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(lane_base + (uint32_t)(h * G::kN + n0 + i)));
            asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(x)::"memory");
            if (hit) x = 0x7FC00000u;
            asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(lane_base + (uint32_t)(h * G::kN + n0 + i)), "r"(x) : "memory");
          }
        }
        tmem_wait_st();
      }
      group_sync(w);  // the part's references, sums and depths are read
      more = more_next;
      if (more && next.n > 0) load_q(next);
      if (!g.empty) {
#pragma unroll 1
        for (int h = 0; h < G::kHalves; ++h) {
          const int d = h * 128 + tk;
#pragma unroll 1
          for (int c = 0; c < kHalf; c += kAtOnce) {
            uint32_t hi[kAtOnce], lo[kAtOnce];
            if (g.n > 0) {
              tmem_cols<kAtOnce>(lane_base + (uint32_t)(h * G::kN + n0 + c), hi);
              tmem_cols<kAtOnce>(lane_base + (uint32_t)(h * G::kN + R + n0 + c), lo);
              tmem_ready<kAtOnce>(hi);
              tmem_ready<kAtOnce>(lo);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
              const int n = n0 + c + i;
              if (m0 + n >= m_all) break;
              const float x = g.n > 0 ? fmaf(__uint_as_float(lo[i]), 0.0625f, __uint_as_float(hi[i])) : 0.f;
              if (g.whole) {
                const int32_t m = (int32_t)(m0 + n), j = fast_div(group_div, m);
                a.out[(int64_t)(g.v.row0 + j) * a.out_stride + (int64_t)(g.kvh * a.group + (m - j * a.group)) * HD + d] =
                    (uint16_t)f32_to_bf16(x * C.inv[n]);
              } else {
                part_o[(part * R + n) * HD + d] = x;
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && g.n > 0) mbar_arrive(sm32(&C.o_free));
      g = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && found.share.n > 0 && (C.abort || !laid_out)) report_error(a.status, kErrTimeout, found.seq);
  if (warp == kC8MmaS)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// Joins the parts of the units that several CTAs share.  A warp has a row of a KV head,
// 4 dims a lane and half, and every kGroups-th part; the groups' results are then added
// in order.  The plan and the parts are written while this launch is already resident, so
// they are no __restrict__ arguments: nothing may read them ahead of the wait.
constexpr int kC8JoinWarps = 8;

template <int HD, int R, int kGroups>
__global__ void __launch_bounds__(32 * kC8JoinWarps)
cache8_join_kernel(const Cache8Args a, const FastDiv group_div, int team_log, int32_t teams, const int64_t *base,
                   const float2 *part_ml, const float4 *part_o, const int32_t *row_seq) {
  constexpr int kQuads = HD / 128;
  __shared__ float4 acc_s[kGroups > 1 ? kC8JoinWarps : 1][kQuads][32];
  __shared__ float2 ml_s[kGroups > 1 ? kC8JoinWarps : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = warp % kGroups;
  const int64_t mg = (int64_t)blockIdx.x * (kC8JoinWarps / kGroups) + warp / kGroups;
  const int32_t kvh = blockIdx.y;
  const int32_t row = mg < (int64_t)a.seqs.n_rows * a.group ? fast_div(group_div, (int32_t)mg) : -1;
  const int32_t head = kvh * a.group + (int32_t)(mg - (int64_t)row * a.group);
  // Where the row lies in the plan, while the launch before still runs: it wrote none of
  // what this reads, and it began after everything before it was complete.
  int32_t s = 0, r = 0, rank = 0, tiles = 0;
  int64_t u0 = 0;  // the unit's first tile, from its sequence's first
  auto place = [&](int32_t at) {  // where the row lies, if sequence `at` has it
    const C8Seq q = c8_seq<R>(a, team_log, read_seq(a.seqs, at));
    if (row < q.v.row0 || row >= q.v.row0 + q.v.rows) return;
    const int64_t m = (int64_t)(row - q.v.row0) * a.group + (head - kvh * a.group);
    const int32_t mt = (int32_t)(m / R);
    s = at;
    r = (int32_t)(m % R);
    rank = mt & ((1 << team_log) - 1);
    tiles = q.tiles;
    u0 = ((int64_t)kvh * q.m_tiles + (mt >> team_log)) * (tiles + kC8Start) + kC8Start;
  };
  if (row >= 0) place(seq_of_row(a.seqs, row));
  grid_dependency_sync();
  // Where bad sequences' starts do not ascend, the search above may have missed a good
  // one: who wrote a part of the row left its sequence.  (A row without parts has what an
  // earlier call left there, which names its sequence or is no place for it.)
  if (row >= 0 && tiles == 0) {
    const int32_t at = row_seq[row];
    if (at >= 0 && at < a.seqs.n_seqs) place(at);
  }
  int32_t c0 = 0, c1 = 0;  // teams of the first and last part
  if (tiles > 0) {
    const int64_t per = (base[a.seqs.n_seqs] + teams - 1) / teams;
    u0 += base[s];
    c0 = (int32_t)(u0 / per);
    c1 = (int32_t)((u0 + tiles - 1) / per);
  }
  const bool mine = c0 != c1;
  float top = -INFINITY, all = 0.f;
  float4 acc[kQuads];
#pragma unroll
  for (int i = 0; i < kQuads; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [](float4 &t, const float4 &x, float by) {
    t.x = fmaf(x.x, by, t.x);
    t.y = fmaf(x.y, by, t.y);
    t.z = fmaf(x.z, by, t.z);
    t.w = fmaf(x.w, by, t.w);
  };
  if (mine) {
    constexpr int kAhead = 4;  // parts on their way
    for (int32_t c = c0 + grp; c <= c1; c += kAhead * kGroups) {
      float2 ml[kAhead];
      float4 x[kAhead][kQuads];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int32_t at = c + e * kGroups;
        const int64_t part = (((int64_t)min(at, c1) << team_log) + rank) * 2 + (min(at, c1) == c0 ? 1 : 0);
        ml[e] = part_ml[part * R + r];
#pragma unroll
        for (int i = 0; i < kQuads; ++i) x[e][i] = part_o[(part * R + r) * (HD / 4) + 32 * i + lane];
        if (at > c1) ml[e] = make_float2(-INFINITY, 0.f);
      }
      float now = top;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) now = fmaxf(now, ml[e].x);
      const float keep = ex2(top - now);  // (a part's reference is finite)
      top = now;
      all *= keep;
#pragma unroll
      for (int i = 0; i < kQuads; ++i) acc[i] = make_float4(acc[i].x * keep, acc[i].y * keep, acc[i].z * keep, acc[i].w * keep);
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        if (ml[e].x == -INFINITY) continue;
        const float by = ex2(ml[e].x - now);
        all = fmaf(ml[e].y, by, all);
#pragma unroll
        for (int i = 0; i < kQuads; ++i) add(acc[i], x[e][i], by);
      }
    }
  }
  if constexpr (kGroups > 1) {
#pragma unroll
    for (int i = 0; i < kQuads; ++i) acc_s[warp][i][lane] = acc[i];
    if (lane == 0) ml_s[warp] = make_float2(top, all);
    __syncthreads();
    if (grp != 0) return;
    for (int g = 1; g < kGroups; ++g) top = fmaxf(top, ml_s[warp + g].x);
    const float use = top == -INFINITY ? 0.f : top;
    all = 0.f;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < kGroups; ++g) {
      if (ml_s[warp + g].x == -INFINITY) continue;
      const float by = ex2(ml_s[warp + g].x - use);
      all = fmaf(ml_s[warp + g].y, by, all);
#pragma unroll
      for (int i = 0; i < kQuads; ++i) add(acc[i], acc_s[warp + g][i][lane], by);
    }
  }
  if (!mine) return;
  const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll
  for (int i = 0; i < kQuads; ++i)
    *reinterpret_cast<uint2 *>(a.out + (int64_t)row * a.out_stride + (int64_t)head * HD + 128 * i + 4 * lane) =
        make_uint2(pack_f32_bf16(acc[i].x * inv, acc[i].y * inv), pack_f32_bf16(acc[i].z * inv, acc[i].w * inv));
  if (lane == 0 && a.lse)
    a.lse[(int64_t)row * a.nq + head] = all == 0.f ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
}

// The workspace: the sequences' first tiles and their sum, the parts' (ref, sum) and O, the
// sequence of each row that has parts.
int64_t rows_of_part(int64_t n_rows, int32_t group) {
  int64_t r = 8;
  while (r < kC8MostRows && r < n_rows * group) r *= 2;
  return r;
}
int64_t base_bytes(int32_t n_seqs) { return ((int64_t)(n_seqs + 1) * 8 + 255) / 256 * 256; }
int64_t ml_bytes(int64_t rows) { return (int64_t)kC8MaxCtas * 2 * rows * 8; }
int64_t o_bytes(int64_t rows, int32_t head_dim) { return (int64_t)kC8MaxCtas * 2 * rows * head_dim * 4; }

template <int HD, int R>
cudaError_t launch_rows(const Cache8Args &a, cudaStream_t stream) {
  static PerDevice smem_attr;
  const cudaError_t e = set_smem_once(smem_attr, cache8_attn_kernel<HD, R>, c8_smem<HD, R>());
  if (e != cudaSuccess) return e;
  uint8_t *ws = static_cast<uint8_t *>(a.ws);
  int64_t *base = reinterpret_cast<int64_t *>(ws);
  float2 *ml = reinterpret_cast<float2 *>(ws + base_bytes(a.seqs.n_seqs));
  float *o = reinterpret_cast<float *>(ws + base_bytes(a.seqs.n_seqs) + ml_bytes(R));
  int32_t *row_seq = reinterpret_cast<int32_t *>(reinterpret_cast<uint8_t *>(o) + o_bytes(R, HD));
  const int64_t mean_rows = (int64_t)a.seqs.n_rows * a.group / a.seqs.n_seqs;
  const int team_log = R < 64 ? 0 : mean_rows >= 224 ? 2 : mean_rows >= 96 ? 1 : 0;
  const int ctas = ((device_sm_count() < kC8MaxCtas ? device_sm_count() : kC8MaxCtas) >> team_log) << team_log;
  const FastDiv group_div = make_fast_div(a.group);
  cudaError_t r = launch_dependent(cache8_attn_kernel<HD, R>, dim3((unsigned)ctas), dim3(kC8Threads), c8_smem<HD, R>(), stream, 1u, a,
                                   group_div, team_log, base, ml, o, row_seq);
  // a table of one tile leaves no unit to share
  if (r != cudaSuccess || (int64_t)a.seqs.table_len * a.seqs.page.d <= kC8T) return r;
  // One group of parts per warp where units outnumber the CTAs (few parts each), eight
  // where a unit spreads over many.
  const int64_t rows = (int64_t)a.seqs.n_rows * a.group, units = (int64_t)a.nkv * ((rows + R - 1) / R);
  const bool many = ctas >= 8 * units;
  return launch_dependent(many ? cache8_join_kernel<HD, R, kC8JoinWarps> : cache8_join_kernel<HD, R, 1>,
                          dim3((unsigned)(many ? rows : (rows + kC8JoinWarps - 1) / kC8JoinWarps), (unsigned)a.nkv),
                          dim3(32 * kC8JoinWarps), 0, stream, 1u, a, group_div, team_log, (int32_t)(ctas >> team_log), base, ml,
                          reinterpret_cast<const float4 *>(o), row_seq);
}

template <int HD>
cudaError_t launch_hd(const Cache8Args &args, cudaStream_t stream) {
  Cache8Args a = args;
  const int64_t most = (int64_t)a.seqs.table_len * a.seqs.page.d;  // (below 2^31 - 256)
  if (a.window >= most) a.window = 0;  // no cached token is that far back
  a.n_first = a.window == 0 ? 0 : (int32_t)(a.n_first < most ? a.n_first : most);
  const int64_t mean_rows = ((int64_t)a.seqs.n_rows * a.group + a.seqs.n_seqs - 1) / a.seqs.n_seqs;
  return mean_rows <= 8    ? launch_rows<HD, 8>(a, stream)
         : mean_rows <= 16 ? launch_rows<HD, 16>(a, stream)
         : mean_rows <= 32 ? launch_rows<HD, 32>(a, stream)
                           : launch_rows<HD, 64>(a, stream);
}

}  // namespace

int64_t cache8_workspace_bytes(int32_t n_seqs, int32_t n_rows, int32_t group, int32_t head_dim) {
  const int64_t rows = rows_of_part(n_rows, group);
  return base_bytes(n_seqs) + ml_bytes(rows) + o_bytes(rows, head_dim) + (int64_t)n_rows * 4;
}

cudaError_t launch_cache8_attn(const Cache8Args &a, int32_t head_dim, cudaStream_t stream) {
  return head_dim == 256 ? launch_hd<256>(a, stream) : launch_hd<128>(a, stream);
}

}  // namespace qsa
