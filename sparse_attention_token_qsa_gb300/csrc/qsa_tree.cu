// Attention of drafted rows over a paged K/V cache.
//
// A sequence has ctx cached tokens and n drafted ones behind them (a tree laid
// out in an order where a parent comes first); drafted row j attends every
// context token and the drafted tokens its mask names:
//   s_t = scale q . k_t,  lse = ln sum_t exp(s_t),  out = sum_t exp(s_t - lse) v_t.
//
// The rows of one sequence that read the same KV head (drafted row x query
// head of the group) form the M dimension of two tcgen05 products per tile of
// 96 tokens (64 at head_dim 256): S = Q K^T (operands in shared memory,
// accumulator in TMEM), and O += P V (P as bf16 in TMEM, V read MN-major).  A unit
// of work is (sequence, KV head, 128 such rows); its tiles are a run of the
// launch's linear list of tiles, of which every CTA (one per SM) takes an equal,
// contiguous share, so ragged batches balance and one long context spreads over
// the GPU.  A unit that lies in one CTA's share is written at once; the parts of
// any other go to the workspace as (O, max, sum) and a second launch joins them in
// a fixed order.
//
// A unit counts kTrStart tiles more than it has, for its Q, its first tile's maximum
// and its output.  At 4, 6, 8 and 12 tiles, 24 sequences of 300 to 9001 tokens with 5 to
// 37 rows of 32 heads over 8 take 115, 112, 111 and 113 us, with 24 rows each 104, 103,
// 104 and 105, with 48 each 164, 159, 159 and 161; 64 single rows over 100 to 2000 tokens
// 94, 91, 93 and 94; 4 sequences of 128 rows over 7k to 16k 115, 114, 116 and 118.
// Where sequences have several tiles of rows, a team of two or four CTAs shares a unit of
// as many: they read the same K and V at the same time, so that these come from HBM
// once.  One by one, in twos and in fours: those 4 sequences (four tiles) 131, 119 and
// 116 us, the 24 with 48 rows (two tiles) 181, 160 and 273, 64 rows of 16 heads over 2
// over 65k tokens 79 each way.  A tile that a team's CTA does not have costs as much as
// one that it has: 24 sequences of 96 rows (three tiles) 268, 313 and 285, and a chunk of
// 512 rows beside 15 single rows over 64k tokens 351, 540 and 988.
//
// Fourteen warps: two groups of four (warps 0-3 and 4-7) do the softmax, a row
// per thread, tiles in turn; warps 8-11 copy K and V rows into a ring of
// slots (a tile of K or of V, 128-byte swizzle); warp 12 issues S, up to three
// tiles ahead, warp 13 P V, so that neither one's waits leave the tensor pipe
// idle.  The copies are 16-byte cp.async, which take any page size alike:
// streaming tiles of pages of 16 tokens and nothing else, they moved 9.7 TB/s
// out of L2 and 5.7 TB/s out of HBM, four-row TMA gathers 5.7 and 4.8, TMA boxes
// of a page 5.5 and 4.6.
//
// The softmax is one pass over a tile's S: the exponentials are taken relative
// to a reference that is a maximum of the row seen earlier, not its running
// maximum.  f32 and bf16 keep their relative precision under any such reference,
// so it only moves (O and the sums rescaled, the tile's pass taken again) when a
// logit passes it by 2^16.  The groups tell each other a row's reference through
// shared memory after each tile; of a group's first tile in a part the first
// columns are passed over beforehand, for a maximum to begin with.
//
// Decode (M = group rows of 128) is bound by HBM: 16 sequences of 16k to 64k tokens take
// 227 us, 94 % of the copy bandwidth.  With more rows no unit is busy all the time: a
// tree of 64 rows over 65471 tokens takes 80 us, 45 % of the bf16 rate, 4 trees of 128
// rows of 32 heads over 8 take 100, 44 %.  A tile's products take 1350 cycles (800 at
// head_dim 128), its copies 2000 (1500) at the 33 bytes a cycle and SM of the probe
// above, its exponentials under 800, and a group's chain of barrier tests (over 100
// cycles each beside the copies), TMEM loads and stores about 3000 for every other tile.
// Measured and no faster: two CTAs as a pair (MMAs of 256 rows, half of each tile a
// CTA), a third softmax group, a second issuer of S, tiles of 128 tokens with fewer
// buffers, K by TMA boxes of 8 tokens, the next unit's Q ahead.
#include "qsa_launch.h"
#include "qsa_paged.cuh"
#include "qsa_tc_cache.cuh"

namespace qsa {

namespace {

constexpr int kTrSoft = 8;     // softmax warps
constexpr int kTrProd = 4;     // producer warps
constexpr int kTrMmaS = kTrSoft + kTrProd;  // issues S = Q K^T
constexpr int kTrMmaO = kTrMmaS + 1;        // issues O += P V
constexpr int kTrWarps = kTrMmaO + 1, kTrThreads = 32 * kTrWarps;
constexpr int kTrRowsLog = 7, kTrRows = 1 << kTrRowsLog;  // rows of a tile: the MMA's M
constexpr int kTrMaxCtas = 160;
constexpr int kTrStart = 8;     // what beginning a unit costs, in tiles
constexpr float kTrSlack = 16.0f;  // log2 units a logit may pass the reference by
constexpr long long kTrSpinLimit = 4000000000LL;

template <int HD>
struct TreeGeom {
  // Tokens per tile: as many as leave TMEM room for three S buffers beside O and P
  // (with two, S of the tile after the next waited for this one's softmax).
  static constexpr int kT = HD == 256 ? 64 : 96;
  static constexpr uint32_t kQBox = kTrRows * 128;          // 64 dims of Q
  static constexpr uint32_t kBox = kT * 128;                // 64 dims of a tile
  static constexpr uint32_t kSlot = kT * HD * 2;            // a ring slot: a tile of K or V
  static constexpr int kSlots = HD == 256 ? 5 : 8;
  static constexpr uint32_t kRingOff = (HD / 64) * kQBox;
  static constexpr uint32_t kCtrlOff = kRingOff + kSlots * kSlot;
  // TMEM columns: O, three S buffers, a P buffer per softmax group
  static constexpr uint32_t kSCol = HD, kPCol = HD + 3 * kT;
  static_assert(kPCol + kT <= 512, "TMEM has 512 columns");
  // kind::f16, D f32, A and B bf16, M = 128; S: N = tokens, K-major B; O: N = dims, MN-major B
  static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);
  static constexpr uint32_t kIdescS = kIdesc | ((uint32_t)(kT >> 3) << 17);
  static constexpr uint32_t kIdescO = kIdesc | ((uint32_t)(HD >> 3) << 17) | (1u << 16);
};

struct TreeCtrl {
  float top[2][kTrRows];   // [group that wrote it][row]: the reference, log2 units
  float sums[2][kTrRows];  // [group][row]: its share of the row's sum
  uint64_t full[8], empty[8];
  uint64_t s_full[3], s_free[3];  // per S buffer: tile % 3
  uint64_t p_ready[2];            // per softmax group
  uint64_t pv_done[4];            // tile % 4
  uint64_t q_full, o_free, drain[2];
  int64_t scan[kTrWarps], found_off;
  int32_t found_seq, bad[2], abort;
  uint32_t tmem_base;
};
template <int HD>
constexpr size_t tree_smem() { return TreeGeom<HD>::kCtrlOff + sizeof(TreeCtrl); }
static_assert(tree_smem<256>() <= 232448 && tree_smem<128>() <= 232448, "227 KiB per CTA");

// What the plan below needs of a sequence.
struct SeqTiles {
  SeqView v;
  int32_t tiles, m_tiles;  // of tokens; of rows, a team's together
  int64_t count;  // tiles of all its units, their starts included
};

template <int T>
__device__ __forceinline__ SeqTiles seq_tiles(const TreeArgs &a, int team_log, const SeqRaw &raw) {
  SeqTiles q;
  q.v = view_seq(a.seqs, raw);
  q.tiles = q.v.rows > 0 ? (q.v.ctx + q.v.rows + T - 1) / T : 0;
  q.m_tiles = (int32_t)(((int64_t)q.v.rows * a.group + (kTrRows << team_log) - 1) >> (kTrRowsLog + team_log));
  q.count = q.tiles > 0 ? (int64_t)(q.tiles + kTrStart) * q.m_tiles * a.nkv : 0;
  return q;
}

// One CTA's part of one unit.
struct TreeSeg {
  int32_t s, kvh, mt;      // sequence, KV head, this CTA's tile of 128 rows
  int32_t t0, n;           // first tile, tiles to process
  bool whole, head;        // the unit's every tile; the unit began in an earlier CTA
  bool empty;              // none of its tiles (a share that ends in a unit's start), or no rows
  SeqView v;
};

// Walks a team's share of the tile list, unit by unit (each role its own walk).
// A sequence's lengths are read one sequence ahead: under load a read takes
// several thousand cycles.
template <int T>
struct TreeWalk {
  const TreeArgs &a;
  int64_t left, off;
  int32_t s;
  int team_log;
  SeqTiles q;
  SeqRaw ahead;
  __device__ TreeWalk(const TreeArgs &a_, int team_log_, int32_t s_, int64_t off_, int64_t left_)
      : a(a_), left(left_), off(off_), s(s_), team_log(team_log_) {
    if (left <= 0) return;
    q = seq_tiles<T>(a, team_log, read_seq(a.seqs, s));
    ahead = read_seq(a.seqs, min(s + 1, a.seqs.n_seqs - 1));
  }
  __device__ bool next(TreeSeg &g) {
    if (left <= 0) return false;
    while (off >= q.count) {
      off -= q.count;
      if (++s >= a.seqs.n_seqs) {
        left = 0;
        return false;
      }
      q = seq_tiles<T>(a, team_log, ahead);
      ahead = read_seq(a.seqs, min(s + 1, a.seqs.n_seqs - 1));
    }
    const int32_t length = q.tiles + kTrStart;
    int32_t unit;  // (KV head, tile of team x 128 rows)
    if ((off >> 31) == 0) unit = (int32_t)((uint32_t)off / (uint32_t)length);
    else unit = (int32_t)(off / length);
    const int32_t from = (int32_t)(off - (int64_t)unit * length);
    const int32_t part = (int32_t)min((int64_t)(length - from), left);
    off += part;
    left -= part;
    g.t0 = max(0, from - kTrStart);
    const int32_t take = max(0, from + part - kTrStart) - g.t0;
    g.s = s;
    g.kvh = unit / q.m_tiles;
    g.mt = ((unit - g.kvh * q.m_tiles) << team_log) + (int32_t)(blockIdx.x & ((1u << team_log) - 1u));
    g.v = q.v;
    g.whole = take == q.tiles;
    g.head = g.t0 > 0;
    g.empty = take == 0 || (int64_t)g.mt * kTrRows >= (int64_t)q.v.rows * a.group;
    g.n = g.empty ? 0 : take;
    if (a.seqs.mask == nullptr && !g.empty) {  // no row of this tile sees past its last row's own token
      const int64_t m_end = min((int64_t)(g.mt + 1) * kTrRows, (int64_t)q.v.rows * a.group);
      const int32_t end = (q.v.ctx + (int32_t)((m_end - 1) / a.group) + T) / T;
      g.n = max(0, min(take, end - g.t0));
    }
    return true;
  }
};

// Ring position of tile j's V among a part's n tiles, counted from the part's
// first copy: K0, K1, V0, K2, V1, ..., V(n-1), about the order the MMAs take them in.
__device__ __forceinline__ int v_pos(int j, int n) { return j + 1 < n ? 2 + 2 * j : 2 * n - 1; }

__device__ __forceinline__ bool nonfinite16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

template <int HD>
__global__ void __launch_bounds__(kTrThreads, 1)
tree_attn_kernel(const TreeArgs a, const FastDiv group_div, int team_log, int32_t part_rows, uint32_t q_and,
                 uint32_t q_xor, int64_t *__restrict__ base_out, float2 *__restrict__ part_ml,
                 float *__restrict__ part_o, int32_t *__restrict__ row_seq) {
  using G = TreeGeom<HD>;
  extern __shared__ __align__(1024) uint8_t tr_smem[];
  TreeCtrl &C = *reinterpret_cast<TreeCtrl *>(tr_smem + G::kCtrlOff);
  const uint32_t sQ = sm32(tr_smem), sRing = sm32(tr_smem + G::kRingOff);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long lim = a.wait_limit > 0 ? a.wait_limit : kTrSpinLimit;
  volatile int32_t *abort_flag = &C.abort;

  if (tid == 0) {
    for (int i = 0; i < G::kSlots; ++i) {
      mbar_init(sm32(&C.full[i]), 32 * kTrProd);
      mbar_init(sm32(&C.empty[i]), 1);
    }
    for (int b = 0; b < 3; ++b) {
      mbar_init(sm32(&C.s_full[b]), 1);
      mbar_init(sm32(&C.s_free[b]), kTrSoft / 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sm32(&C.p_ready[b]), kTrSoft / 2);
      mbar_init(sm32(&C.drain[b]), 1);
      C.bad[b] = 0;
    }
    for (int b = 0; b < 4; ++b) mbar_init(sm32(&C.pv_done[b]), 1);
    mbar_init(sm32(&C.q_full), 32 * kTrSoft);
    mbar_init(sm32(&C.o_free), kTrSoft);
    C.abort = 0;
    C.found_seq = a.seqs.n_seqs;
    C.found_off = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  grid_dependency_sync();  // before TMEM too: an earlier launch may hold it
  if (warp == kTrMmaS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     sm32(&C.tmem_base)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- the plan: every sequence's tiles summed, then the sequence this CTA's
  // share starts in (CTA 0 also leaves the sums for the joining launch).  Up to 32
  // sequences, a lane each, every warp for itself; else a thread each, in chunks.
  int64_t total = 0, found_off = 0;
  int32_t found_seq = a.seqs.n_seqs;
  TileShare share = {0, 0, 0};
  const uint32_t teams = gridDim.x >> team_log, my_team = blockIdx.x >> team_log;
  auto tiles_of = [&](int32_t s, bool report) -> int64_t {
    if (s >= a.seqs.n_seqs) return 0;
    const SeqTiles q = seq_tiles<G::kT>(a, team_log, read_seq(a.seqs, s));
    if (report && !q.v.ok) report_error(a.status, kErrRowRange, s);
    return q.count;
  };
  if (a.seqs.n_seqs <= 32) {
    const bool writes = blockIdx.x == 0 && warp == 0;
    const int64_t count = tiles_of(lane, writes), incl = warp_scan(count, lane), at = incl - count;
    total = __shfl_sync(0xffffffffu, incl, 31);
    share = tile_share(total, teams, my_team);
    if (writes && lane < a.seqs.n_seqs) base_out[lane] = at;
    const uint32_t hit = __ballot_sync(0xffffffffu, share.n > 0 && count > 0 && at <= share.first && share.first < incl);
    if (hit != 0) {
      found_seq = __ffs(hit) - 1;
      found_off = share.first - __shfl_sync(0xffffffffu, at, found_seq);
    }
  } else {
    const bool one_chunk = a.seqs.n_seqs <= kTrThreads;
    if (!one_chunk) {
      for (int32_t s = tid; s < a.seqs.n_seqs; s += kTrThreads) total += tiles_of(s, false);
      for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      if (lane == 0) C.scan[warp] = total;
      __syncthreads();
      total = 0;
      for (int i = 0; i < kTrWarps; ++i) total += C.scan[i];
    }
    int64_t before = 0;
    for (int32_t s0 = 0; s0 < a.seqs.n_seqs; s0 += kTrThreads) {
      const int32_t s = s0 + tid;
      const int64_t count = tiles_of(s, blockIdx.x == 0), incl = warp_scan(count, lane);
      __syncthreads();
      if (lane == 31) C.scan[warp] = incl;
      __syncthreads();
      int64_t at = before + incl - count;
#pragma unroll
      for (int i = 0; i < kTrWarps; ++i) {
        at += i < warp ? C.scan[i] : 0;
        before += C.scan[i];
      }
      if (one_chunk) total = before;
      share = tile_share(total, teams, my_team);
      if (s < a.seqs.n_seqs && blockIdx.x == 0) base_out[s] = at;
      if (share.n > 0 && count > 0 && at <= share.first && share.first < at + count) {
        C.found_seq = s;
        C.found_off = share.first - at;
      }
      if (blockIdx.x != 0 && before > share.first) break;
    }
  }
  if (blockIdx.x == 0 && tid == 0) base_out[a.seqs.n_seqs] = total;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem_base;
  const bool laid_out = (sQ & 1023u) == 0;  // the swizzle needs it; the declaration asks for it
  if (a.seqs.n_seqs > 32) {
    found_seq = C.found_seq;
    found_off = C.found_off;
  }
  TreeWalk<G::kT> walk(a, team_log, found_seq, found_off, laid_out ? share.n : 0);
  TreeSeg g;

  if (warp >= kTrSoft && warp < kTrMmaS) {
    // ---- producers: warp p brings a quarter of each tile's tokens, 512 bytes an
    // instruction (kRows rows); lane i looks up the pool row of its i-th token.  A
    // slot's barrier takes each thread's arrival when its copies have landed, so the
    // whole ring may be in flight.
    constexpr int kCh = HD / 8, kRows = 32 / kCh, kTok = G::kT / kTrProd, kN = kTok / kRows;
    const int p0 = (warp - kTrSoft) * kTok, ch = lane % kCh, hl = lane / kCh;
    const uint32_t dst0 = sRing + (uint32_t)(ch >> 3) * G::kBox + (uint32_t)(p0 + hl) * 128u;
    uint32_t ns = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      const int32_t kv = g.v.ctx + g.v.rows;
      auto fetch = [&](int j) -> int32_t {  // pool row of this lane's token of tile j, -1: zeros
        const int32_t t = (g.t0 + j) * G::kT + p0 + lane;
        if (j >= g.n || t >= kv || lane >= kTok) return -1;
        const int64_t slot = token_slot(a.seqs, g.s, t);
        if (slot < 0) report_error(a.status, kErrTokenRange, g.s);
        return slot < 0 ? -1 : (int32_t)(slot * a.nkv + g.kvh);
      };
      // Pool rows of this thread's copies of a slot, spread from the lanes that
      // looked them up before the slot is waited for: a shuffle between the copies
      // of a slot cost 90 cycles a copy.
      auto spread = [&](int32_t y, int32_t (&r)[kN]) {
#pragma unroll
        for (int k = 0; k < kN; ++k) r[k] = __shfl_sync(0xffffffffu, y, kRows * k + hl);
      };
      auto bring = [&](const uint16_t *pool, const int32_t (&r)[kN]) {
        const uint32_t slot = ns % G::kSlots;
        if (!tc_warp_wait_ready(sm32(&C.empty[slot]), ((ns / G::kSlots) & 1u) ^ 1u, lim, abort_flag)) {
          ok = false;
          return;
        }
        __syncwarp();
        const uint16_t *src = pool + ch * 8;
#pragma unroll
        for (int k = 0; k < kN; ++k)  // row p0 + kRows k + hl, its 16-byte chunks swizzled by row % 8
          cp_async16(dst0 + slot * G::kSlot + (uint32_t)(k * kRows) * 128u +
                         (uint32_t)(((ch & 7) ^ ((kRows * k + hl) & 7)) << 4),
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
      if (warp == kTrSoft && !g.whole && !g.empty) {  // the rows of a part, for the join
        const int64_t m0 = (int64_t)g.mt * kTrRows, m1 = min(m0 + kTrRows, (int64_t)g.v.rows * a.group);
        const int32_t end = fast_div(group_div, (int32_t)m1 - 1);
        for (int32_t j = fast_div(group_div, (int32_t)m0) + lane; j <= end; j += 32) row_seq[g.v.row0 + j] = g.s;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives the CTA
  } else if (warp >= kTrMmaS) {
    // ---- MMA issuers, one thread each.  What they do between MMAs is on the tensor
    // pipe's time, so slots, buffers and phases are stepped, not divided.
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
      // before this one has to be known to have landed.  S of tile j (five slots; more
      // are easier): that one is K, of a tile whose S this thread issued, or V of tile
      // j - 4 at the latest, whose P V was waited for, or, where j begins a part, the
      // last V of a part before the last, whose output was written before this part's
      // Q was fetched.  P V of tile j: it is V, or K of an earlier tile.
      auto landed = [&]() {
        if (!wait(C.full[slot], phase)) return false;
        // the copies wrote through the generic proxy; the MMAs read through the async one
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_after();
        return true;
      };
      // A descriptor's address sits in its low word: the steps of a tile add to it
      // (shared memory ends below 2^18, so no carry leaves the address's 14 bits).
      const uint32_t desc_hi = (uint32_t)(sw128_desc(0) >> 32);
      uint32_t jg = 0, part = 0;  // tiles and parts before this one
      if (warp == kTrMmaS) {
        const uint32_t q_lo = (uint32_t)sw128_desc(sQ), r_lo = (uint32_t)sw128_desc(sRing);
        uint32_t b = 0, b_phase = 1;  // S buffer, parity of its s_free phase before this use
        while (ok && walk.next(g)) {
          if (g.n == 0) continue;
          if (!wait(C.q_full, part & 1u)) break;
          ++part;
          for (int j = 0; j < g.n; ++j, ++jg) {
            if (jg >= 3 && !wait(C.s_free[b], b_phase)) break;  // tile j - 3 is read
            if (HD == 256 && jg >= 4 && !wait(C.pv_done[jg & 3u], ((jg >> 2) & 1u) ^ 1u)) break;
            if (j > 0) step(j == 1 ? 1u : 2u);
            if (!landed()) break;
            const uint32_t d = tmem + G::kSCol + b * G::kT, k_lo = r_lo + slot * (G::kSlot >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint32_t in = (uint32_t)(kk & 3) * 2u;  // 32 bytes
              mma_bf16(d, desc_of(q_lo + (uint32_t)(kk >> 2) * (G::kQBox >> 4) + in, desc_hi),
                       desc_of(k_lo + (uint32_t)(kk >> 2) * (G::kBox >> 4) + in, desc_hi), G::kIdescS, kk > 0 ? 1u : 0u);
            }
            mma_commit(sm32(&C.empty[slot]));
            mma_commit(sm32(&C.s_full[b]));
            if (++b == 3) {
              b = 0;
              b_phase ^= 1u;
            }
          }
          step(g.n == 1 ? 2u : 3u);  // past V(n - 2) and V(n - 1)
        }
      } else {
        const uint32_t r_lo = (uint32_t)sw128_mn_desc(sRing, G::kBox);
        while (ok && walk.next(g)) {
          if (g.n == 0) continue;
          if (part > 0 && !wait(C.o_free, (part - 1) & 1u)) break;  // the part before has left O
          ++part;
          for (int j = 0; j < g.n; ++j, ++jg) {
            if (!wait(C.p_ready[jg & 1u], (jg >> 1) & 1u)) break;
            step(j + 1 < g.n ? 2u : 1u);
            if (!landed()) break;
            const uint32_t p = tmem + G::kPCol + (jg & 1u) * (G::kT / 2), v_lo = r_lo + slot * (G::kSlot >> 4);
#pragma unroll
            for (int kk = 0; kk < G::kT / 16; ++kk)  // 16 tokens a step: 8 columns of P, 2 KiB of a V box
              mma_bf16_ts(tmem, p + 8u * kk, desc_of(v_lo + 128u * kk, desc_hi), G::kIdescO, (j > 0 || kk > 0) ? 1u : 0u);
            mma_commit(sm32(&C.empty[slot]));
            mma_commit(sm32(&C.pv_done[jg & 3u]));
          }
          step(1u);
        }
      }
      // every MMA this thread issued has finished before TMEM is freed
      mma_commit(sm32(&C.drain[warp - kTrMmaS]));
      tc_wait(sm32(&C.drain[warp - kTrMmaS]), 0u, kTrSpinLimit, nullptr);
    }
    __syncwarp();
  } else {
    // ---- softmax: thread = TMEM lane (row) r of group w; the groups take the
    // CTA's tiles in turn and half of the output's dims each.  After an abort every
    // wait returns at once, and the loops and the pairs' barriers run on to the end.
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // a row's maximum from one group to the other: barrier 1 + warp (0..7) of the
    // sender, which arrives, while the warp of the same rows waits
    auto post = [&](float x) {
      C.top[w][r] = x;
      asm volatile("bar.arrive %0, 64;" ::"r"(1 + warp) : "memory");
    };
    auto receive = [&]() -> float {
      asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp ^ 4)) : "memory");
      return C.top[w ^ 1][r];
    };
    // P V of tile i.  A group has waited for tile i - 4 (or a later one) by then,
    // so of a barrier no phase but the last two is ever in question.
    auto wait_pv = [&](uint32_t i) {
      tc_warp_wait_ready(sm32(&C.pv_done[i & 3u]), (i >> 2) & 1u, lim, abort_flag);
    };
    // This warp's rows of a part's Q into shared memory.  The copies arrive on
    // q_full by themselves; a sign or a zero scale has to pass through registers, and the
    // arrival of a thread's copies would not wait for its stores: it arrives behind them.
    auto load_q = [&](const TreeSeg &e) {
      const int64_t m0 = (int64_t)e.mt * kTrRows;
      const int rows = (int)min((int64_t)kTrRows, (int64_t)e.v.rows * a.group - m0);
      constexpr int kCh = HD / 8;     // 16-byte chunks per row
      constexpr int kPer = 32 / kCh;  // rows per warp copy
      const int ch = lane % kCh, sub = lane / kCh;
      const bool plain = q_and == 0xFFFFFFFFu && q_xor == 0u;
#pragma unroll 4
      for (int rr = warp * kPer + sub; rr < rows; rr += kPer * kTrSoft) {
        const int32_t m = (int32_t)(m0 + rr), j = fast_div(group_div, m);
        const int32_t head = e.kvh * a.group + (m - j * a.group);
        const uint16_t *src = a.q + (int64_t)(e.v.row0 + j) * a.q_stride + (int64_t)head * HD + 8 * ch;
        const uint32_t to = (uint32_t)(ch >> 3) * G::kQBox + (uint32_t)rr * 128u + (uint32_t)(((ch & 7) ^ (rr & 7)) << 4);
        if (plain) {
          cp_async16(sQ + to, src, 16u);
        } else {
          uint4 v = *reinterpret_cast<const uint4 *>(src);
          v.x = (v.x & q_and) ^ q_xor;
          v.y = (v.y & q_and) ^ q_xor;
          v.z = (v.z & q_and) ^ q_xor;
          v.w = (v.w & q_and) ^ q_xor;
          *reinterpret_cast<uint4 *>(tr_smem + to) = v;
        }
      }
      if (plain) cp_async_arrive(sm32(&C.q_full));
      else mbar_arrive(sm32(&C.q_full));
    };
    uint32_t jg = 0, ns = 0;
    int32_t seg = 0;
    const uint64_t c2 = pair_f32(a.scale_log2, a.scale_log2);
    bool more = walk.next(g);
    if (more && g.n > 0) load_q(g);
    while (more) {
      ++seg;
      const int64_t m = (int64_t)g.mt * kTrRows + r;
      const bool valid = m < (int64_t)g.v.rows * a.group;
      const bool live = __any_sync(0xffffffffu, valid);  // this warp (and its pair) has rows
      const int32_t j_row = valid ? fast_div(group_div, (int32_t)m) : 0;
      const int32_t row = g.v.row0 + j_row;
      const int32_t head = g.kvh * a.group + (valid ? (int32_t)m - j_row * a.group : 0);
      const uint32_t *mrow = a.seqs.mask ? a.seqs.mask + (int64_t)row * a.seqs.mask_words : nullptr;
      // whether a row may be blind to a token that another one sees
      const bool veiled = g.v.rows > 1 || a.seqs.mask != nullptr;
      TreeSeg next;
      const bool more_next = walk.next(next);  // while the first S is on its way
      float top = -INFINITY, sum = 0.f;  // sum is relative to top
      auto rebase = [&](float t) {
        if (t != top) {
          sum *= top == -INFINITY ? 0.f : ex2(top - t);  // (a NaN so far stays)
          top = t;
        }
      };
      for (int j = 0; j < g.n; ++j, ++jg) {
        if ((int)(jg & 1u) != w) continue;
        const uint32_t b = jg % 3u, sc = lane_base + G::kSCol + b * G::kT, pc = lane_base + G::kPCol + (uint32_t)w * (G::kT / 2);
        const int32_t t0 = (g.t0 + j) * G::kT;
        const bool masked = t0 + G::kT > g.v.ctx;
        tc_warp_wait_ready(sm32(&C.s_full[b]), (jg / 3u) & 1u, lim, abort_flag);
        tc_fence_after();
        if (live) {
          uint64_t see[(G::kT + 63) / 64];
          if (masked) {
#pragma unroll
            for (int i = 0; i < (G::kT + 63) / 64; ++i)
              see[i] = sees64(mrow, a.seqs.mask_words, j_row, g.v.rows, t0 + 64 * i - g.v.ctx);
          }
          // probe: for a maximum alone, of the first columns that a row sees any of
          bool probe = j < 2, told = j == 0;  // told: of what the tile before left
          float t = -INFINITY;
          float part;
          while (true) {
            const float use = top == -INFINITY ? 0.f : top;
            const uint64_t m2 = pair_f32(-use, -use);
            uint64_t part2[2] = {0ull, 0ull};
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < G::kT / 32; ++c) {
              uint32_t sv[32];
              tmem_ld32(sc + 32u * c, sv);
              tmem_wait_ld32(sv);
              if (masked) {
                const uint32_t bits = (uint32_t)(see[c >> 1] >> (32 * (c & 1)));
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!((bits >> i) & 1u)) sv[i] = 0xFF800000u;  // -inf
              }
#pragma unroll
              for (int i = 0; i < 16; ++i)
                mx[i & 1] = max3(mx[i & 1], __uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
              if (probe) {
                if (__all_sync(0xffffffffu, !valid || fmaxf(mx[0], mx[1]) != -INFINITY)) break;
              } else {
                uint32_t p[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float lo, hi;
                  unpair_f32(fma2(pair_f32(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), c2, m2), lo, hi);
                  lo = ex2(lo);
                  hi = ex2(hi);
                  // The sums keep 32 bits, as lse has to; P is rounded to bf16, the type
                  // that the MMA takes beside V's.  Each weight is then off by half a
                  // bf16 step at most, as the output is by its own rounding: 0.0023 of
                  // the output's norm against 64 bits, 0.0017 if P had 32 bits.
                  part2[i & 1] = add2(part2[i & 1], pair_f32(lo, hi));
                  p[i] = pack_f32_bf16(lo, hi);
                }
                if (c == 0 && jg >= 2) {  // P's buffer is free
                  wait_pv(jg - 2);
                  tc_fence_after();
                }
                tmem_st16(pc + 16u * c, p);
              }
            }
            float s0, s1;
            unpair_f32(add2(part2[0], part2[1]), s0, s1);
            part = s0 + s1;
            // what the other group's tile left, and whether this one passes it
            if (!told) t = receive();
            told = true;
            const float mine = fmaxf(mx[0], mx[1]);
            const float want = mine == -INFINITY ? -INFINITY : mine * a.scale_log2;
            const bool move = valid && (want > t + kTrSlack || (t == -INFINITY && want != -INFINITY));
            const float now = move ? want : t;
            if (!__any_sync(0xffffffffu, probe || now != top)) break;
            if (j > 0 && __any_sync(0xffffffffu, move)) {  // O holds the earlier tiles of this part
              const float alpha = move ? (t == -INFINITY ? 0.f : ex2(t - now)) : 1.f;
              wait_pv(jg - 1);
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < HD / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(lane_base + (uint32_t)(c * 16), o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st16(lane_base + (uint32_t)(c * 16), o);
              }
              tmem_wait_st();
            }
            rebase(now);
            t = now;
            probe = false;
          }
          post(top);
          sum += part;
          tmem_wait_st();
        } else if (jg >= 2) {
          wait_pv(jg - 2);  // every warp keeps up with the barriers
        }
        if (masked && veiled) {
          // A value that is not finite would reach, as 0 x inf, the rows that do
          // not see its token: it is cleared here and given to the rows that do
          // see it when the output is written.  (The slot's earlier copy is known to
          // have landed once P V of the tile before the last is done.)
          {
            const uint32_t at = ns + (uint32_t)v_pos(j, g.n), slot = at % G::kSlots;
            tc_warp_wait_ready(sm32(&C.full[slot]), (at / G::kSlots) & 1u, lim, abort_flag);
            __syncwarp();
            uint8_t *vs = tr_smem + G::kRingOff + slot * G::kSlot;
            const int first = max(0, g.v.ctx - t0), n = min(G::kT, g.v.ctx + g.v.rows - t0) - first;
            for (int i = (warp & 3) * 32 + lane; i < n * (HD / 8); i += 128) {  // 16 bytes, in no order that matters
              const int row = first + i / (HD / 8), ch = i % (HD / 8);
              uint4 *q = reinterpret_cast<uint4 *>(vs + (ch >> 3) * G::kBox + row * 128 + (ch & 7) * 16);
              const uint4 x = *q;
              uint32_t e[4] = {x.x, x.y, x.z, x.w};
              bool hit = false;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (nonfinite16(e[k])) { e[k] &= 0xFFFF0000u; hit = true; }
                if (nonfinite16(e[k] >> 16)) { e[k] &= 0xFFFFu; hit = true; }
              }
              if (hit) {
                *q = make_uint4(e[0], e[1], e[2], e[3]);
                *reinterpret_cast<volatile int32_t *>(&C.bad[seg & 1]) = seg;
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(sm32(&C.s_free[b]));
          mbar_arrive(sm32(&C.p_ready[w]));
        }
      }
      ns += (uint32_t)(2 * g.n);
      const uint32_t last = jg - 1;  // the part's last tile
      if (g.n > 0) {  // its S is done, and with it every one of this part: Q may go
        tc_warp_wait_ready(sm32(&C.s_full[last % 3u]), (last / 3u) & 1u, lim, abort_flag);
        __syncwarp();
        if (live && (int)(last & 1u) != w) rebase(receive());
      }
      more = more_next;
      if (more && next.n > 0) load_q(next);
      if (g.n > 0) {
        if (last > 0 && (int)(last & 1u) != w) wait_pv(last - 1);
        wait_pv(last);
        tc_fence_after();
      }
      if (live && !g.empty) {
        C.sums[w][r] = sum;
        asm volatile("bar.sync %0, 64;" ::"r"(9 + (warp & 3)) : "memory");
        const float all = C.sums[0][r] + C.sums[1][r];
        asm volatile("bar.sync %0, 64;" ::"r"(9 + (warp & 3)) : "memory");  // read before the next part's
        const float inv = all == 0.f ? 0.f : 1.f / all;
        const bool fix = *reinterpret_cast<volatile int32_t *>(&C.bad[seg & 1]) == seg;
        const int64_t part = (int64_t)blockIdx.x * 2 + (g.head ? 0 : 1);
        if (valid && w == 0) {
          if (!g.whole) part_ml[part * part_rows + r] = make_float2(top, all);
          else if (a.lse) a.lse[(int64_t)row * a.nq + head] =
              all == 0.f ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
        }
#pragma unroll 1
        for (int c = 0; c < HD / 64; ++c) {
          const int d0 = w * (HD / 2) + c * 32;
          uint32_t o[32];
          __syncwarp();
          if (g.n > 0) {
            tmem_ld32(lane_base + (uint32_t)d0, o);
            tmem_wait_ld32(o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (!valid) continue;
          if (fix) {
            // every drafted token of this part
            const int32_t t_lo = max(g.t0 * G::kT, g.v.ctx);
            const int32_t t_hi = min(g.v.ctx + g.v.rows, (g.t0 + g.n) * G::kT);
            for (int32_t t = t_lo; t < t_hi; ++t) {
              if (!sees_draft(mrow, j_row, t - g.v.ctx)) continue;
              const int64_t slot = token_slot(a.seqs, g.s, t);
              if (slot < 0) continue;
              const uint16_t *v = a.v_pool + (slot * a.nkv + g.kvh) * HD + d0;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (nonfinite16(v[i])) o[i] = __float_as_uint(__uint_as_float(o[i]) + bf16_to_f32(v[i]));
            }
          }
          if (g.whole) {
            uint16_t *dst = a.out + (int64_t)row * a.out_stride + (int64_t)head * HD + d0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_f32_bf16(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
              reinterpret_cast<uint4 *>(dst)[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            // [dims / 4][row] quads: a warp's rows lie side by side
            uint4 *dst = reinterpret_cast<uint4 *>(part_o) + (part * (HD / 4) + d0 / 4) * part_rows + r;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i * part_rows] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && g.n > 0) mbar_arrive(sm32(&C.o_free));
      g = next;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && share.n > 0 && (C.abort || !laid_out)) report_error(a.status, kErrTimeout, found_seq);
  if (warp == kTrMmaS)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// Joins the parts of the units that several CTAs share.  A warp takes 8 rows x 4
// times kQuads quads of dims (a part's rows lie side by side) and every
// kGroups-th part, two at a time with the running maximum: one trip to L2 for both
// the maxima and the values.  The groups' results are then added in order.
// The plan and the parts are written while this launch is already resident, so they
// are no __restrict__ arguments: nothing may read them ahead of the wait, or as if no
// one wrote them.
constexpr int kJoinWarps = 8;

template <int HD, int kGroups, int kQuads>
__global__ void __launch_bounds__(32 * kJoinWarps)
tree_join_kernel(const TreeArgs a, const FastDiv group_div, int team_log, int32_t part_rows, int32_t teams,
                 const int64_t *base, const float2 *part_ml, const float4 *part_o, const int32_t *row_seq) {
  __shared__ float4 acc_s[kGroups > 1 ? kJoinWarps : 1][kQuads][32];
  __shared__ float2 ml_s[kGroups > 1 ? kJoinWarps : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp % kGroups;
  const int64_t mg = ((int64_t)blockIdx.x * (kJoinWarps / kGroups) + warp / kGroups) * 8 + (lane & 7);
  const int32_t quad = blockIdx.y * (4 * kQuads) + (lane >> 3), kvh = blockIdx.z;
  const int32_t row = mg < (int64_t)a.seqs.n_rows * a.group ? fast_div(group_div, (int32_t)mg) : -1;
  const int32_t head = kvh * a.group + (int32_t)(mg - (int64_t)row * a.group);
  // Where the row lies in the plan, while the launch before still runs: it wrote none
  // of what this reads, and it began after everything before it was complete.
  int32_t s = 0, r = 0, rank = 0, tiles = 0;
  int64_t u0 = 0;  // the unit's first tile, from its sequence's first
  auto place = [&](int32_t at) {  // where the row lies, if sequence `at` has it
    const SeqTiles q = seq_tiles<TreeGeom<HD>::kT>(a, team_log, read_seq(a.seqs, at));
    if (row < q.v.row0 || row >= q.v.row0 + q.v.rows) return;
    const int64_t m = (int64_t)(row - q.v.row0) * a.group + (head - kvh * a.group);
    const int32_t mt = (int32_t)(m >> kTrRowsLog);
    s = at;
    r = (int32_t)(m & (kTrRows - 1));
    rank = mt & ((1 << team_log) - 1);
    tiles = q.tiles;
    u0 = ((int64_t)kvh * q.m_tiles + (mt >> team_log)) * (tiles + kTrStart) + kTrStart;
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
    if (((u0 + tiles) >> 31) == 0) {
      c0 = (int32_t)((uint32_t)u0 / (uint32_t)per);
      c1 = (int32_t)((uint32_t)(u0 + tiles - 1) / (uint32_t)per);
    } else {
      c0 = (int32_t)(u0 / per);
      c1 = (int32_t)((u0 + tiles - 1) / per);
    }
  }
  const bool mine = c0 != c1;
  auto part_of = [&](int32_t c) { return (((int64_t)c << team_log) + rank) * 2 + (c == c0 ? 1 : 0); };
  const float2 none = make_float2(-INFINITY, 0.f);
  float top = -INFINITY, all = 0.f;
  float4 acc[kQuads];
#pragma unroll
  for (int i = 0; i < kQuads; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [](float4 &s, const float4 &x, float w) {
    s.x = fmaf(x.x, w, s.x);
    s.y = fmaf(x.y, w, s.y);
    s.z = fmaf(x.z, w, s.z);
    s.w = fmaf(x.w, w, s.w);
  };
  auto scaled = [](const float4 &x, float w) { return make_float4(x.x * w, x.y * w, x.z * w, x.w * w); };
  if (mine) {
    for (int32_t c = c0 + grp; c <= c1; c += 2 * kGroups) {
      float2 ml[2];
      float4 x[2][kQuads];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool there = e == 0 || c + kGroups <= c1;
        const int64_t part = part_of(there ? c + e * kGroups : c);
        ml[e] = there ? part_ml[part * part_rows + r] : none;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
          x[e][i] = there ? part_o[(part * (HD / 4) + quad + 4 * i) * part_rows + r] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      const float now = fmaxf(top, fmaxf(ml[0].x, ml[1].x)), use = now == -INFINITY ? 0.f : now;
      const float w = ex2(top - use), w0 = ex2(ml[0].x - use), w1 = ex2(ml[1].x - use);
      top = now;
      all = fmaf(ml[1].y, w1, fmaf(ml[0].y, w0, all * w));
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        acc[i] = scaled(acc[i], w);
        add(acc[i], x[0][i], w0);
        add(acc[i], x[1][i], w1);
      }
    }
  }
  if constexpr (kGroups > 1) {
#pragma unroll
    for (int i = 0; i < kQuads; ++i) acc_s[warp][i][lane] = acc[i];
    ml_s[warp][lane] = make_float2(top, all);
    __syncthreads();
    if (grp != 0) return;
    for (int g = 1; g < kGroups; ++g) top = fmaxf(top, ml_s[warp + g][lane].x);
    const float use = top == -INFINITY ? 0.f : top;
    all = 0.f;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float w = ex2(ml_s[warp + g][lane].x - use);
      all = fmaf(ml_s[warp + g][lane].y, w, all);
#pragma unroll
      for (int i = 0; i < kQuads; ++i) add(acc[i], acc_s[warp + g][i][lane], w);
    }
  }
  if (!mine) return;
  const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll
  for (int i = 0; i < kQuads; ++i)
    *reinterpret_cast<uint2 *>(a.out + (int64_t)row * a.out_stride + (int64_t)head * HD + 4 * (quad + 4 * i)) =
        make_uint2(pack_f32_bf16(acc[i].x * inv, acc[i].y * inv), pack_f32_bf16(acc[i].z * inv, acc[i].w * inv));
  if (quad == 0 && a.lse)
    a.lse[(int64_t)row * a.nq + head] = all == 0.f ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
}

// The workspace: the sequences' first tiles and their sum, the parts' (max, sum) and O, the
// sequence of each row that has parts.
int32_t part_rows_of(int64_t n_rows, int32_t group) {
  return (int32_t)(n_rows * group < kTrRows ? n_rows * group : kTrRows);
}
int64_t base_bytes(int32_t n_seqs) { return ((int64_t)(n_seqs + 1) * 8 + 255) / 256 * 256; }
int64_t o_bytes(int32_t part_rows, int32_t head_dim) { return (int64_t)kTrMaxCtas * 2 * part_rows * head_dim * 4; }
int64_t ml_bytes(int32_t part_rows) { return ((int64_t)kTrMaxCtas * 2 * part_rows * 8 + 255) / 256 * 256; }

template <int HD>
cudaError_t launch_hd(const TreeArgs &args, cudaStream_t stream) {
  static PerDevice smem_attr;
  const cudaError_t e = set_smem_once(smem_attr, tree_attn_kernel<HD>, tree_smem<HD>());
  if (e != cudaSuccess) return e;
  TreeArgs a = args;
  // the kernel takes scale > 0: a negative one turns q's signs, a zero one clears q
  uint32_t q_and = 0xFFFFFFFFu, q_xor = 0u;
  if (a.scale_log2 < 0.f) {
    a.scale_log2 = -a.scale_log2;
    q_xor = 0x80008000u;
  } else if (a.scale_log2 == 0.f) {
    a.scale_log2 = 1.f;
    q_and = 0u;
  }
  const int32_t part_rows = part_rows_of(a.seqs.n_rows, a.group);
  uint8_t *ws = static_cast<uint8_t *>(a.ws);
  int64_t *base = reinterpret_cast<int64_t *>(ws);
  float2 *ml = reinterpret_cast<float2 *>(ws + base_bytes(a.seqs.n_seqs));
  float *o = reinterpret_cast<float *>(ws + base_bytes(a.seqs.n_seqs) + ml_bytes(part_rows));
  int32_t *row_seq = reinterpret_cast<int32_t *>(reinterpret_cast<uint8_t *>(o) + o_bytes(part_rows, HD));
  // CTAs that take a unit's tiles of rows side by side: from one and a half tiles a
  // sequence on two, from three and a half four.  The lengths are the device's, so the
  // host goes by the mean over the call (measured both ways at the head of this file).
  const int64_t mean_rows = (int64_t)a.seqs.n_rows * a.group / a.seqs.n_seqs;
  const int team_log = mean_rows >= 448 ? 2 : mean_rows >= 192 ? 1 : 0;
  const int ctas = ((device_sm_count() < kTrMaxCtas ? device_sm_count() : kTrMaxCtas) >> team_log) << team_log;
  const FastDiv group_div = make_fast_div(a.group);
  cudaError_t r = launch_dependent(tree_attn_kernel<HD>, dim3((unsigned)ctas), dim3(kTrThreads), tree_smem<HD>(), stream, 1u,
                                   a, group_div, team_log, part_rows, q_and, q_xor, base, ml, o, row_seq);
  // a table of one tile leaves no unit to share
  if (r != cudaSuccess || (int64_t)a.seqs.table_len * a.seqs.page.d <= TreeGeom<HD>::kT) return r;
  // One group of parts per warp where units outnumber the CTAs (few parts each),
  // eight where a unit spreads over many.
  const int64_t rows8 = ((int64_t)a.seqs.n_rows * a.group + 7) / 8;
  const int64_t units = (int64_t)a.nkv * (((int64_t)a.seqs.n_rows * a.group + kTrRows - 1) / kTrRows);
  const bool many = ctas >= 8 * units;
  const int64_t blocks = many ? rows8 : (rows8 + kJoinWarps - 1) / kJoinWarps;
  // Four quads a thread keep more reads on their way where blocks come in waves (64
  // rows of 65k tokens: 79.8 us, 82.9 with one); one where they are few (12.0 us for a
  // row of 515 tokens, 12.9 with four).
  const bool few = many && rows8 * a.nkv * (HD / 16) <= device_sm_count();
  return launch_dependent(few    ? tree_join_kernel<HD, kJoinWarps, 1>
                          : many ? tree_join_kernel<HD, kJoinWarps, 4>
                                 : tree_join_kernel<HD, 1, 4>,
                          dim3((unsigned)blocks, few ? HD / 16 : HD / 64, (unsigned)a.nkv), dim3(32 * kJoinWarps), 0, stream, 1u, a,
                          group_div, team_log, part_rows, (int32_t)(ctas >> team_log), base, ml, reinterpret_cast<const float4 *>(o),
                          row_seq);
}

}  // namespace

int64_t tree_workspace_bytes(int32_t n_seqs, int32_t n_rows, int32_t group, int32_t head_dim) {
  const int32_t rows = part_rows_of(n_rows, group);
  return base_bytes(n_seqs) + ml_bytes(rows) + o_bytes(rows, head_dim) + (int64_t)n_rows * 4;
}

cudaError_t launch_tree_attn(const TreeArgs &a, int32_t head_dim, cudaStream_t stream) {
  return head_dim == 256 ? launch_hd<256>(a, stream) : launch_hd<128>(a, stream);
}

}  // namespace qsa
