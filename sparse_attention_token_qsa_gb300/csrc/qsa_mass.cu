// The attention weight that cached tokens gather.
//
// For KV head g of a sequence, token t's mass becomes
//   carry * mass[t] + sum_r w_r sum_{h in g} exp(scale q_rh . k_t - lse_rh)
// over the drafted rows r that see t; a drafted token's mass starts at zero.
//
// Keys are the M dimension of one tcgen05 product per tile of 128 tokens: S^T = K
// Q^T with the (row, head) pairs on N, so a thread that reads its TMEM lane holds
// one token's logits, adds up their exponentials in registers (no maximum is
// needed, lse is given) and owns the token's mass: no atomics, and a sum's order is
// that of the rows.  Up to 128 or 256 pairs' Q stay in shared memory while K
// streams through a ring of slots (128 tokens x 64 or 128 dims) of 16-byte
// cp.async copies; more pairs are taken in turns, K read again from L2.  Rows of
// weight 0 are left out of Q.
//
// Every CTA (one per SM) takes an equal, contiguous share of the launch's list of
// (sequence, KV head, tile), in which beginning a (sequence, KV head) counts as some
// tiles more.  Fourteen warps: warps 0-3 and 4-7 sum a tile in turn, warps 8-11 copy
// K, warp 12 issues the MMAs, warp 13 walks the share and names the rows of each turn.
//
// With few pairs the kernel is bound by reading K once from HBM: 16 sequences of
// 16k to 64k tokens, a row of 16 heads over 2 each, take 104 us, 85 % of the copy
// bandwidth.  With many: 64 rows of the same heads over 65471 tokens take 42 us.  The
// products alone would take 18 (M128 N256 K16 in 128 cycles); a turn begins with 4000
// cycles for its Q (128 KiB at the rate L2 gives an SM), and a tile's sums wait for
// one another's latency (TMEM load, exponential).  Four groups, two to a tile, took 45.
// The plan counts a tile once, however many turns pass over it: sequences of very unequal
// rows in one call leave the wide one's tiles to few CTAs (a chunk of 512 rows beside 15
// single rows over 64k tokens: 3.1 ms, 0.17 and 0.22 in two calls).
#include <type_traits>

#include "qsa_launch.h"
#include "qsa_paged.cuh"
#include "qsa_tc_cache.cuh"

namespace qsa {

namespace {

constexpr int kMsSum = 8, kMsProd = 4;
constexpr int kMsMma = kMsSum + kMsProd, kMsPlan = kMsMma + 1;
constexpr int kMsWarps = kMsPlan + 1, kMsThreads = 32 * kMsWarps;
constexpr int kMsT = 128;                  // tokens per tile: the MMA's M
constexpr int kMsQueue = 2;
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596303e-8f;  // log2(e) in two words
constexpr uint32_t kMsBox = kMsT * 128;    // 64 dims of a tile: 16 KiB
constexpr long long kMsSpinLimit = 4000000000LL;

template <int HD, int NR>
struct MassGeom {
  static constexpr int kB = HD == 256 && NR == 256 ? 1 : 2;  // 64-dim boxes per slot
  static constexpr int kC = HD / (64 * kB);                  // slots per tile
  static constexpr uint32_t kSlot = kB * kMsBox;
  static constexpr uint32_t kQBox = NR * 128;
  static constexpr uint32_t kRingOff = (HD / 64) * kQBox;
  // What beginning a (sequence, KV head) costs, in tiles: its turns' pairs and Q, its
  // masked tile.  3 sequences of 15k to 25k tokens with 33 to 40 rows of 32 heads over 8:
  // 41 us without, 39.4 at 2, 38.5 at 3 and 4; 6 of 2k to 5k: 35, 32.8, 31.5, 35; 20 of
  // 500 to 3000 with 1 to 4 rows: 14.3 without, 14.1 at 1, 13.4 at 2.
  static constexpr int kStart = NR == 256 ? 3 : 2;
  static constexpr int kSlots = HD == 256 ? 5 : (NR == 256 ? 4 : 6);
  static constexpr uint32_t kCtrlOff = kRingOff + kSlots * kSlot;
};

// A turn: tiles [t0, t0 + n) of one (sequence, KV head) against up to NR (row,
// head) pairs, the first of them head h0 of the listed rows' first.
struct MassTurn {
  int32_t n, t0, s, kvh;  // n = -1: the share's end
  int32_t row0, rows, ctx;
  int32_t cols, h0, first;
};

template <int NR>
struct MassCtrl {
  float4 colv[NR / 2];          // per two pairs: -lse in log2 units, weights
  int32_t list[kMsQueue][NR + 2];  // the turn's rows, as offsets from row0
  uint64_t full[6], empty[6];
  uint64_t s_full[2], s_free[2];
  uint64_t q_full, cv_full, turn_done, drain;
  uint64_t turn_full[kMsQueue], turn_empty[kMsQueue];
  MassTurn turn[kMsQueue];
  int64_t scan[kMsWarps], found_off;
  int32_t found_seq, abort;
  int32_t dull[2];  // [turn parity]: the turn (from 1) some pair of which adds nothing
  uint32_t tmem_base;
};
template <int HD, int NR>
constexpr size_t mass_smem() { return MassGeom<HD, NR>::kCtrlOff + sizeof(MassCtrl<NR>); }
static_assert(mass_smem<256, 256>() <= 232448 && mass_smem<256, 128>() <= 232448 &&
                  mass_smem<128, 256>() <= 232448 && mass_smem<128, 128>() <= 232448, "227 KiB per CTA");

struct MassSeq {
  SeqView v;
  int32_t tiles;
  int64_t count;
};

template <class G>
__device__ __forceinline__ MassSeq mass_seq(const MassArgs &a, int32_t s) {
  MassSeq q;
  q.v = view_seq(a.seqs, s);
  if (q.v.ok && (int64_t)q.v.ctx + q.v.rows > a.mass_cols) {
    q.v.ok = false;
    q.v.rows = 0;
  }
  q.tiles = q.v.rows > 0 ? (q.v.ctx + q.v.rows + kMsT - 1) / kMsT : 0;
  q.count = q.tiles > 0 ? (int64_t)(q.tiles + G::kStart) * a.nkv : 0;
  return q;
}

template <int HD, int NR>
__global__ void __launch_bounds__(kMsThreads, 1)
attn_mass_kernel(const MassArgs a, const FastDiv group_div, float c, float c_rel) {
  using G = MassGeom<HD, NR>;
  extern __shared__ __align__(1024) uint8_t ms_smem[];
  MassCtrl<NR> &C = *reinterpret_cast<MassCtrl<NR> *>(ms_smem + G::kCtrlOff);
  const uint32_t sQ = sm32(ms_smem), sRing = sm32(ms_smem + G::kRingOff);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long lim = a.wait_limit > 0 ? a.wait_limit : kMsSpinLimit;
  volatile int32_t *abort_flag = &C.abort;

  if (tid == 0) {
    for (int i = 0; i < G::kSlots; ++i) {
      mbar_init(sm32(&C.full[i]), 32 * kMsProd);
      mbar_init(sm32(&C.empty[i]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sm32(&C.s_full[b]), 1);
      mbar_init(sm32(&C.s_free[b]), kMsSum / 2);
    }
    for (int b = 0; b < kMsQueue; ++b) {
      mbar_init(sm32(&C.turn_full[b]), 1);
      mbar_init(sm32(&C.turn_empty[b]), kMsPlan);  // every warp before the planner
    }
    mbar_init(sm32(&C.q_full), 32 * kMsSum);
    mbar_init(sm32(&C.cv_full), kMsSum);
    mbar_init(sm32(&C.turn_done), kMsSum);
    mbar_init(sm32(&C.drain), 1);
    C.abort = 0;
    C.dull[0] = C.dull[1] = 0;
    C.found_seq = a.seqs.n_seqs;
    C.found_off = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  grid_dependency_sync();  // before TMEM too: an earlier launch may hold it
  if (warp == kMsMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     sm32(&C.tmem_base)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- the plan: every sequence's tiles summed, then the sequence this CTA's
  // share starts in.  Up to 32 sequences, a lane each, every warp for itself; else a
  // thread each, in chunks.
  int64_t total = 0, found_off = 0;
  int32_t found_seq = a.seqs.n_seqs;
  TileShare part = {0, 0, 0};
  auto tiles_of = [&](int32_t s, bool report) -> int64_t {
    if (s >= a.seqs.n_seqs) return 0;
    const MassSeq q = mass_seq<G>(a, s);
    if (report && !q.v.ok) report_error(a.status, kErrRowRange, s);
    return q.count;
  };
  if (a.seqs.n_seqs <= 32) {
    const int64_t count = tiles_of(lane, blockIdx.x == 0 && warp == 0), incl = warp_scan(count, lane), at = incl - count;
    total = __shfl_sync(0xffffffffu, incl, 31);
    part = tile_share(total, gridDim.x, blockIdx.x);
    const uint32_t hit = __ballot_sync(0xffffffffu, part.n > 0 && count > 0 && at <= part.first && part.first < incl);
    if (hit != 0) {
      found_seq = __ffs(hit) - 1;
      found_off = part.first - __shfl_sync(0xffffffffu, at, found_seq);
    }
  } else {
    const bool one_chunk = a.seqs.n_seqs <= kMsThreads;
    if (!one_chunk) {
      for (int32_t s = tid; s < a.seqs.n_seqs; s += kMsThreads) total += tiles_of(s, false);
      for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      if (lane == 0) C.scan[warp] = total;
      __syncthreads();
      total = 0;
      for (int i = 0; i < kMsWarps; ++i) total += C.scan[i];
    }
    int64_t before = 0;
    for (int32_t s0 = 0; s0 < a.seqs.n_seqs; s0 += kMsThreads) {
      const int32_t s = s0 + tid;
      const int64_t count = tiles_of(s, blockIdx.x == 0), incl = warp_scan(count, lane);
      __syncthreads();
      if (lane == 31) C.scan[warp] = incl;
      __syncthreads();
      int64_t at = before + incl - count;
#pragma unroll
      for (int i = 0; i < kMsWarps; ++i) {
        at += i < warp ? C.scan[i] : 0;
        before += C.scan[i];
      }
      if (one_chunk) total = before;
      part = tile_share(total, gridDim.x, blockIdx.x);
      if (part.n > 0 && count > 0 && at <= part.first && part.first < at + count) {
        C.found_seq = s;
        C.found_off = part.first - at;
      }
      if (blockIdx.x != 0 && before > part.first) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem_base;
  if (a.seqs.n_seqs > 32) {
    found_seq = C.found_seq;
    found_off = C.found_off;
  }
  const bool laid_out = (sQ & 1023u) == 0;  // the swizzle needs it; the declaration asks for it

  // The next turn of the share (a whole warp, or the issuer's one thread).
  uint32_t qn = 0;
  bool ok = laid_out && part.n > 0;  // (a CTA without a share has nothing to wait for)
  auto take_turn = [&](MassTurn &g, bool one_thread) -> bool {
    const uint32_t e = qn % kMsQueue, par = (qn / kMsQueue) & 1u;
    ok = ok && (one_thread ? tc_wait_ready(sm32(&C.turn_full[e]), par, lim, abort_flag)
                           : tc_warp_wait_ready(sm32(&C.turn_full[e]), par, lim, abort_flag));
    if (!ok) return false;
    if (!one_thread) __syncwarp();
    g = C.turn[e];
    ++qn;
    return g.n >= 0;
  };
  auto done_turn = [&](bool one_thread) {  // with the entry taken last, and its list
    if (!one_thread) __syncwarp();
    if (one_thread || lane == 0) mbar_arrive(sm32(&C.turn_empty[(qn - 1) % kMsQueue]));
  };

  if (warp == kMsPlan) {
    // ---- the share's turns: rows of weight 0 are passed over
    int64_t left = part.n, off = found_off;
    int32_t s = found_seq;
    auto push = [&](const MassTurn &g) {  // (the list is written)
      __syncwarp();
      if (lane == 0) {
        C.turn[qn % kMsQueue] = g;
        mbar_arrive(sm32(&C.turn_full[qn % kMsQueue]));
      }
      ++qn;
    };
    auto room = [&]() {
      const uint32_t e = qn % kMsQueue;
      ok = ok && tc_warp_wait_ready(sm32(&C.turn_empty[e]), ((qn / kMsQueue) & 1u) ^ 1u, lim, abort_flag);
      __syncwarp();
      return ok;
    };
    while (left > 0 && ok) {
      MassSeq q = mass_seq<G>(a, s);
      while (off >= q.count) {
        off -= q.count;
        if (++s >= a.seqs.n_seqs) break;
        q = mass_seq<G>(a, s);
      }
      if (s >= a.seqs.n_seqs) break;  // (a share ends inside the last sequence)
      MassTurn g;
      g.s = s;
      const int32_t length = q.tiles + G::kStart;
      g.kvh = (off >> 31) == 0 ? (int32_t)((uint32_t)off / (uint32_t)length) : (int32_t)(off / length);
      const int32_t from = (int32_t)(off - (int64_t)g.kvh * length), run = (int32_t)min((int64_t)(length - from), left);
      g.t0 = max(0, from - G::kStart);
      g.n = max(0, from + run - G::kStart) - g.t0;
      off += run;
      left -= run;
      if (g.n == 0) continue;  // a share that ends in a start
      g.row0 = q.v.row0;
      g.rows = q.v.rows;
      g.ctx = q.v.ctx;
      g.first = 1;
      g.h0 = 0;
      int32_t j = 0, last = 0;  // next row to look at; the row that the turn before cut
      auto weigh = [&](int32_t jj) { return a.weight && jj < g.rows ? a.weight[g.row0 + jj] : 1.f; };
      float ahead = weigh(lane);  // of row j + lane
      while (room()) {
        int32_t *list = C.list[qn % kMsQueue];
        int32_t found = 0;
        if (g.h0 > 0) {
          if (lane == 0) list[0] = last;
          found = 1;
        }
        while (j < g.rows && (int64_t)found * a.group - g.h0 < NR) {
          const int32_t jj = j + lane;
          const bool on = jj < g.rows && ahead != 0.f;
          const float next = weigh(jj + 32);
          const uint32_t bits = __ballot_sync(0xffffffffu, on);
          const int32_t want = (NR + g.h0 - found * a.group + a.group - 1) / a.group;  // rows still fitting
          const int32_t rank = __popc(bits & ((1u << lane) - 1u));
          if (on && rank < want) list[found + rank] = jj;
          if (__popc(bits) >= want) {  // stop behind the last row taken
            const uint32_t at = __ballot_sync(0xffffffffu, on && rank == want - 1);
            j += __ffs(at);
            last = j - 1;
            found += want;
            ahead = weigh(j + lane);
          } else {
            if (bits) last = j + 31 - __clz(bits);
            j += 32;
            found += __popc(bits);
            ahead = next;
          }
        }
        const int64_t have = (int64_t)found * a.group - g.h0;
        g.cols = (int32_t)min((int64_t)NR, have);
        if (g.cols == 0 && !g.first) break;
        push(g);
        const bool cut = have > NR;
        g.h0 = cut ? a.group - (int32_t)(have - NR) : 0;
        g.first = 0;
        if (!cut && j >= g.rows) break;
      }
    }
    if (ok && room()) {
      MassTurn g;
      g.n = -1;
      push(g);
    }
  } else if (warp >= kMsSum && warp < kMsMma) {
    // ---- producers: warp p brings tokens 32p .. 32p + 31 of each tile's K, 512
    // bytes (kRows rows of a slot) an instruction; lane i looks up the pool row of
    // its token.
    constexpr int kCh = 8 * G::kB, kRows = 32 / kCh, kN = 32 / kRows;
    const int p0 = (warp - kMsSum) * 32, ch = lane % kCh, hl = lane / kCh;
    const uint32_t dst0 = sRing + (uint32_t)(ch >> 3) * kMsBox + (uint32_t)(p0 + hl) * 128u;
    uint32_t slot = 0, phase = 1;
    MassTurn g;
    while (take_turn(g, false)) {
      done_turn(false);
      if (g.cols == 0) continue;
      auto fetch = [&](int j) -> int32_t {  // pool row of this lane's token of tile j, -1: zeros
        const int32_t t = (g.t0 + j) * kMsT + p0 + lane;
        if (j >= g.n || t >= g.ctx + g.rows) return -1;
        const int64_t at = token_slot(a.seqs, g.s, t);
        if (at < 0) report_error(a.status, kErrTokenRange, g.s);
        return at < 0 ? -1 : (int32_t)(at * a.nkv + g.kvh);
      };
      int32_t y = fetch(0);
      for (int j = 0; j < g.n && ok; ++j) {
        int32_t r[kN];
#pragma unroll
        for (int k = 0; k < kN; ++k) r[k] = __shfl_sync(0xffffffffu, y, kRows * k + hl);
        y = fetch(j + 1);
#pragma unroll
        for (int c = 0; c < G::kC; ++c) {
          ok = ok && tc_warp_wait_ready(sm32(&C.empty[slot]), phase, lim, abort_flag);
          if (!ok) break;
          __syncwarp();
          const uint16_t *src = a.k_pool + c * (64 * G::kB) + ch * 8;
#pragma unroll
          for (int k = 0; k < kN; ++k)  // row p0 + kRows k + hl, its 16-byte chunks swizzled by row % 8
            cp_async16(dst0 + slot * G::kSlot + (uint32_t)(k * kRows) * 128u +
                           (uint32_t)(((ch & 7) ^ ((kRows * k + hl) & 7)) << 4),
                       src + (int64_t)max(r[k], 0) * HD, r[k] >= 0 ? 16u : 0u);
          cp_async_arrive(sm32(&C.full[slot]));
          if (++slot == (uint32_t)G::kSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives the CTA
  } else if (warp == kMsMma) {
    // ---- MMA issuer (one thread): S^T of a tile, N = the turn's pairs rounded up to 16
    if (lane == 0) {
      auto wait = [&](uint64_t &bar, uint32_t parity) {
        ok = ok && tc_wait_ready(sm32(&bar), parity, lim, abort_flag);
        return ok;
      };
      const uint32_t desc_hi = (uint32_t)(sw128_desc(0) >> 32);
      const uint32_t q_lo = (uint32_t)sw128_desc(sQ), r_lo = (uint32_t)sw128_desc(sRing);
      uint32_t slot = 0, phase = 0, jg = 0, turn = 0;
      MassTurn g;
      while (take_turn(g, true)) {
        done_turn(true);
        if (g.cols == 0) continue;
        // kind::f16, D f32, A and B bf16, both K-major, M = 128
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)((g.cols + 15) >> 4) << 18) | ((128u >> 4) << 24);
        if (!wait(C.q_full, turn & 1u)) break;
        ++turn;
        for (int j = 0; j < g.n; ++j, ++jg) {
          const uint32_t b = jg & 1u, d = tmem + b * NR;
          if (jg >= 2 && !wait(C.s_free[b], ((jg >> 1) - 1u) & 1u)) break;
#pragma unroll
          for (int c = 0; c < G::kC; ++c) {
            if (!wait(C.full[slot], phase)) break;
            // the copies wrote through the generic proxy; the MMAs read through the async one
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_after();
            const uint32_t k_lo = r_lo + slot * (G::kSlot >> 4);
#pragma unroll
            for (int kk = 0; kk < 4 * G::kB; ++kk) {
              const uint32_t in = (uint32_t)(kk & 3) * 2u;
              mma_bf16(d, desc_of(k_lo + (uint32_t)(kk >> 2) * (kMsBox >> 4) + in, desc_hi),
                       desc_of(q_lo + (uint32_t)(G::kB * c + (kk >> 2)) * (G::kQBox >> 4) + in, desc_hi), idesc,
                       (c > 0 || kk > 0) ? 1u : 0u);
            }
            mma_commit(sm32(&C.empty[slot]));
            if (++slot == (uint32_t)G::kSlots) {
              slot = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          mma_commit(sm32(&C.s_full[b]));
        }
        if (!ok) break;
      }
      // every MMA this thread issued has finished before TMEM is freed
      mma_commit(sm32(&C.drain));
      tc_wait(sm32(&C.drain), 0u, kMsSpinLimit, nullptr);
    }
    __syncwarp();
  } else {
    // ---- sums: thread = TMEM lane = token r of the tiles its group takes
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(w * NR);
    const uint64_t c2 = pair_f32(c, c);
    auto wait = [&](uint64_t &bar, uint32_t parity) {
      ok = ok && tc_warp_wait_ready(sm32(&bar), parity, lim, abort_flag);
      return ok;
    };
    uint32_t jg = 0, turn = 0, seen = 0;
    MassTurn g;
    while (take_turn(g, false)) {
      const int32_t *list = C.list[(qn - 1) % kMsQueue];
      // ---- the turn's Q and what belongs to its pairs, once the turn before is over
      if (seen > 0 && !wait(C.turn_done, (seen - 1) & 1u)) break;
      __syncwarp();
      ++seen;
      const int cols16 = (g.cols + 15) & ~15;
      if (g.cols > 0) {
        constexpr int kCh = HD / 8, kPer = 32 / kCh;  // 16-byte chunks a row, rows a warp copy
        const int ch = lane % kCh, sub = lane / kCh;
#pragma unroll 8
        for (int f = warp * kPer + sub; f < cols16; f += kPer * kMsSum) {
          const uint32_t to = sQ + (uint32_t)(ch >> 3) * G::kQBox + (uint32_t)f * 128u + (uint32_t)(((ch & 7) ^ (f & 7)) << 4);
          const uint16_t *src = a.q;
          if (f < g.cols) {
            const int32_t i = fast_div(group_div, f + g.h0);
            src += (int64_t)(g.row0 + list[i]) * a.q_stride + (int64_t)(g.kvh * a.group + f + g.h0 - i * a.group) * HD + 8 * ch;
          }
          cp_async16(to, src, f < g.cols ? 16u : 0u);
        }
        cp_async_arrive(sm32(&C.q_full));
        const int f = warp * 32 + lane;  // one pair a thread
        if (f < cols16) {
          float2 v = make_float2(INFINITY, 0.f);  // what adds nothing
          if (f < g.cols) {
            const int32_t i = fast_div(group_div, f + g.h0);
            const int64_t row = g.row0 + list[i];
            const float lse = a.lse[row * a.nq + g.kvh * a.group + f + g.h0 - i * a.group];
            if (lse != -INFINITY) {
              // exp(scale s - lse) = 2^(s c - l): what c and l lose to f32 goes into the
              // weight, c's share at s c = l, where the token that matters lies.  l is
              // the product of lse and log2(e), the latter in two words; its f32
              // rounding and the rest are exact but for the rest's own rounding.
              v.x = __fmul_rn(lse, kLog2eHi);
              const float rest = fmaf(lse, kLog2eHi, -v.x) + lse * kLog2eLo;
              const float lost = fmaf(c_rel, v.x, -rest);  // log2 units, under 2^-22 of l
              const float w = a.weight ? a.weight[row] : 1.f;
              v.y = lost == lost ? fmaf(w, 0.69314718f * lost, w) : w;
            }
          }
          float *at = reinterpret_cast<float *>(&C.colv[f >> 1]) + (f & 1);
          at[0] = -v.x;
          at[2] = v.y;
          if (v.x == INFINITY) *reinterpret_cast<volatile int32_t *>(&C.dull[turn & 1u]) = (int32_t)turn + 1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sm32(&C.cv_full));
        if (!wait(C.cv_full, turn & 1u)) break;
        __syncwarp();
        ++turn;
      }
      // pairs that add nothing (padding, lse -inf) must not add NaN for a key that is
      // not finite either
      const bool dull = *reinterpret_cast<volatile int32_t *>(&C.dull[(turn - 1) & 1u]) == (int32_t)turn;
      float *mass = a.mass + ((int64_t)g.s * a.nkv + g.kvh) * a.mass_cols;
      for (int j = 0; j < g.n && ok; ++j) {
        // (a turn without pairs only scales: no tile of it is multiplied)
        const uint32_t at = g.cols > 0 ? jg + (uint32_t)j : (uint32_t)j;
        if ((int)(at & 1u) != w) continue;
        const int32_t t0 = (g.t0 + j) * kMsT, t = t0 + r;
        const bool in = t < g.ctx + g.rows;
        float old = 0.f;
        if (in && (g.first ? t < g.ctx && a.carry != 0.f : true)) old = mass[t];
        float sum = 0.f;
        if (g.cols > 0) {
          if (!wait(C.s_full[w], (at >> 1) & 1u)) break;
          tc_fence_after();
          const bool masked = t0 + kMsT > g.ctx;
          const int32_t k0 = t0 + (warp & 3) * 32 - g.ctx;  // drafted index of the warp's first token
          uint64_t acc[2] = {0ull, 0ull};
          // 16 pairs from c on; `plain`: every one counts for every token
          auto add = [&](auto plain, const uint32_t *sv, int c) {
            uint32_t sees = 0;
            int i0 = 0;
            if (!plain.value) asm volatile("" : "+r"(c));
            if (!plain.value && masked) {
              const int last_row = (int)fast_div(group_div, g.cols - 1 + g.h0);
              // lane i: which of the warp's 32 tokens the i-th row of these pairs sees
              i0 = fast_div(group_div, c + g.h0);
              if (i0 + lane <= last_row && lane < 16) {
                const int32_t jr = list[i0 + lane];
                sees = (uint32_t)sees64(a.seqs.mask ? a.seqs.mask + (int64_t)(g.row0 + jr) * a.seqs.mask_words : nullptr,
                                        a.seqs.mask_words, jr, g.rows, k0);
              }
            }
            const float4 *cv = C.colv + c / 2;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 v = cv[i];
              float lo, hi;
              unpair_f32(fma2(pair_f32(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), c2, pair_f32(v.x, v.y)),
                         lo, hi);
              if (!plain.value) {
                if (v.x == -INFINITY) lo = -INFINITY;
                if (v.y == -INFINITY) hi = -INFINITY;
                if (masked) {
                  const uint32_t s0 = __shfl_sync(0xffffffffu, sees, fast_div(group_div, c + 2 * i + g.h0) - i0);
                  const uint32_t s1 = __shfl_sync(0xffffffffu, sees, fast_div(group_div, c + 2 * i + 1 + g.h0) - i0);
                  if (!((s0 >> lane) & 1u)) lo = -INFINITY;
                  if (!((s1 >> lane) & 1u)) hi = -INFINITY;
                }
              }
              acc[i & 1] = fma2(pair_f32(ex2(lo), ex2(hi)), pair_f32(v.z, v.w), acc[i & 1]);
            }
          };
          auto sweep = [&](auto plain) {
            int c = 0;
            for (; c + 32 <= cols16; c += 32) {
              uint32_t sv[32];
              __syncwarp();
              tmem_ld32(lane_base + (uint32_t)c, sv);
              tmem_wait_ld32(sv);
              add(plain, sv, c);
              add(plain, sv + 16, c + 16);
            }
            if (c < cols16) {
              uint32_t sv[16];
              __syncwarp();
              tmem_ld16(lane_base + (uint32_t)c, sv);
              add(plain, sv, c);
            }
          };
          if (masked || dull) sweep(std::false_type{});
          else sweep(std::true_type{});
          float s0, s1;
          unpair_f32(add2(acc[0], acc[1]), s0, s1);
          sum = s0 + s1;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(sm32(&C.s_free[w]));
        }
        if (in) mass[t] = g.first ? fmaf(a.carry, old, sum) : old + sum;
      }
      if (!ok) break;
      if (g.cols > 0) jg += (uint32_t)g.n;
      // Both groups have seen the turn's last S, so Q may go: a group that did not
      // take that tile waits for it too.
      if (g.cols > 0 && (int)((jg - 1) & 1u) != w && !wait(C.s_full[(jg - 1) & 1u], ((jg - 1) >> 1) & 1u)) break;
      done_turn(false);
      if (lane == 0) mbar_arrive(sm32(&C.turn_done));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && part.n > 0 && (C.abort || !laid_out)) report_error(a.status, kErrTimeout, found_seq);
  if (warp == kMsMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <int HD, int NR>
cudaError_t launch_mass(const MassArgs &a, cudaStream_t stream) {
  static PerDevice smem_attr;
  const cudaError_t e = set_smem_once(smem_attr, attn_mass_kernel<HD, NR>, mass_smem<HD, NR>());
  if (e != cudaSuccess) return e;
  // the logits' factor in log2 units, and what its f32 rounding lost, relative to it
  const double scale_log2 = (double)a.scale * 1.4426950408889634;
  const float c = (float)scale_log2;
  const float c_rel = scale_log2 != 0.0 ? (float)((scale_log2 - (double)c) / scale_log2) : 0.f;
  return launch_dependent(attn_mass_kernel<HD, NR>, dim3((unsigned)device_sm_count()), dim3(kMsThreads),
                          mass_smem<HD, NR>(), stream, 1u, a, make_fast_div(a.group), c, c_rel);
}

}  // namespace

cudaError_t launch_attn_mass(const MassArgs &a, int32_t head_dim, cudaStream_t stream) {
  // 256 pairs a turn halve what many rows read of K again; 128 leave shared memory
  // for a deeper ring, which reading K once from HBM needs.  A sequence of 65k tokens with
  // 64, 128, 160 and 512 pairs: 16, 20, 29 and 67 us with 128, 19, 22, 24 and 56 with 256;
  // four of 12k with 96, 128, 192 and 512: 30, 33, 54 and 113 against 29, 33, 41 and 91.
  const bool many = (int64_t)a.seqs.n_rows * a.group > (int64_t)128 * a.seqs.n_seqs;
  if (head_dim == 256) return many ? launch_mass<256, 256>(a, stream) : launch_mass<256, 128>(a, stream);
  return many ? launch_mass<128, 256>(a, stream) : launch_mass<128, 128>(a, stream);
}

}  // namespace qsa
