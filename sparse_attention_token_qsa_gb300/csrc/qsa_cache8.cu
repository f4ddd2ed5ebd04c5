// Attention over a paged cache held in 8 bits, with a scale for each block of tokens and
// head, and with a window over the tokens that a row looks back at.
//
//   s_t = scale ks_t q . k8_t,  lse = ln sum_t exp(s_t),  out = sum_t exp(s_t - lse) vs_t v8_t
//
// over the tokens t that the row sees.  The products run on tcgen05 in 8 bits, the type the
// cache is held in, straight from the tiles that the copies leave in shared memory:
// nothing is widened.  Tokens are the M dimension: a tile of 128 gives S^T = K Q^T (lanes
// tokens, columns rows) and O^T += V^T P (lanes dims, columns rows, V and P read MN-major).
// So a tile of 8 rows costs an MMA of N = 16, not one padded to 128 rows, a thread has one
// token and with it one K and one V scale, and a row's reference moves with its columns.
//
// What few bits lose is kept in further terms, their own columns beside the first.  q 2^-e = hi +
// lo / 16, both e4m3: a bf16 q has eight bits, so this is off by 2^-21 of the head's largest
// value and exact where q is 2^-13 of it or more.  The weight w = exp(s - ref) vs = hi + (mid +
// lo) / 4, all e5m2 (P's type; V's stays e4m3): off by 2^-9 of itself and 2^-11 for its passage
// through f16, or by 2^-19.  ref is log2 of a maximum of exp(s) vs seen earlier, less 8, so that
// is 2^-27 of the row's largest.  Many small weights may still outweigh one that is larger, as
// beside a first token whose V is small (with two e4m3 terms, 2^-18, the outputs of 65536 tokens
// beside one of weight 0.9 were off by 14 to 27 % of their norm): a maximum that is more than 10
// binades above the others of its tile is put up to 6 higher.  ref moves (the row's sum and its columns of
// O rescaled) when a w passes 57344, e5m2's largest: a move costs most of a tile's time, and the
// 7.8 binades before it are why 8 and not more (8, 10, 11, 12, 14: 64 rows of 65k tokens 107,
// 109, 116, 126, 138 us, a chunk of 2048 in a window 168, 185, 202, 213, 236).  The sum is of the
// f32 weights without vs.  Against 64 bits the outputs are off by 0.0017 of their norm, as with q
// and weights of 32 bits: bf16's rounding.
//
// A unit of work is (sequence, KV head, R such rows); its tiles are a run of the launch's
// linear list of tiles, of which every CTA (one per SM) takes an equal, contiguous share.
// A unit that lies in one CTA's share is written at once; the parts of any other go to
// the workspace as (O, ref, sum) and a second launch joins them in a fixed order.  CTAs take
// up to eight KV heads side by side: they read neighbouring pieces of the same rows at the
// same time, which for 8 heads of 128 bytes brought HBM from 5.3 to 6.4 TB/s.  Units of
// rows side by side gained nothing (64 rows of 65k tokens 126 us each way) and lost where
// sequences have fewer units (24 of 5 to 37 rows 194 us alone, 227 in pairs).
//
// Roles by warp: groups of four do the softmax, a token of a tile per thread; four copy K
// and V rows into a ring of slots (16-byte cp.async, 128-byte swizzle); one issues S, one
// P V; one looks pages up, ahead, and brings the scales; one walks the CTA's share and hands
// its parts to the others.  Their loops run side by side and share one instruction cache:
// at about 40 KB of hot code a quarter of the fetches missed, and every instruction waited three
// cycles for its fetch (decode 118 us, 64 rows of 65k 197 us); one copy loop, waits of a few
// instructions and MMAs issued from a uniform loop took the misses to 5 % (106 and 127 us).
// For the same reason a part's beginning and end are short: they run once or twice a launch.
// (Where they run often, they bound it: 512 rows over 64 to 400 tokens of 8 KV heads, 27 parts
// of one to four tiles a CTA, take 118 us, 4.4 us a part.)
//
// Decode is bound by HBM: 16 sequences of 16k to 64k tokens, 16 heads over 2 x 256, take
// 102 us, 93 % of the copy bandwidth; 32 heads over 8 x 128 193 us, 99 %.  With more rows the
// softmax bounds it: a tile of 64 rows is 8192 weights and 8300 warp instructions of all roles,
// 32 for every 32 weights, most of them a softmax warp's: S's two terms joined, two scales, the
// exponential, the sum, three terms of w, and beside its 16 columns what a tile costs each of
// the 16 warps (barriers, votes, look-ups).  64 rows of 65471 tokens take 107 us (34 % of the
// bf16 rate), the MMAs busy for 36 % of it and 59 % of the issue slots used.
#include "qsa_launch.h"
#include "qsa_share.cuh"
#include "qsa_tc_cache.cuh"

namespace qsa {

namespace {

constexpr int kC8Prod = 4;  // warps that copy
constexpr int kC8Segs = 4;  // parts that the walk is ahead by
constexpr int kC8T = 128;        // tokens of a tile: the MMAs' M
constexpr int kC8MostRows = 64;  // rows of a unit at most
constexpr int kC8MaxCtas = 160;
constexpr float kC8Unset = -1e30f;    // a row's reference before it has seen a token
constexpr float kC8Nobody = 1e30f;    // ... of a column without a row: its weights are 0
constexpr float kC8Head = 8.f;        // log2 of a largest w when the reference is set
constexpr float kC8Gap = 10.f;        // ... and more by what it is above the others beyond this,
constexpr float kC8Lift = 6.f;        // up to this
constexpr float kC8Most = 57344.f;    // a w above moves the reference: e5m2's largest
constexpr float kC8Least = 0x1p-80f;  // a V scale below counts as this for the reference
constexpr uint32_t kC8SuspendNs = 2000;  // a wait's sleep at most (it ends early when its phase completes)
constexpr long long kC8SpinLimit = 4000000000LL;

template <int HD, int R>
struct C8Geom {
  static constexpr int kN = 2 * R;               // columns: hi terms, lo terms
  static constexpr int kHalves = HD / 128;
  // Up to 32 rows two softmax groups of four warps take tiles in turn, each with a sum,
  // references and an O of its own, joined at the part's end; of 64, four groups take a
  // quarter of every tile's rows each.  (Two groups with a half of them: a chunk of 2048 rows
  // in a window of 1024 229 us, four 207 then; trees of 5 to 37 rows 176 and 169; 64 rows of 65k
  // tokens 116 each way.  Two that take tiles of 64 columns in turn, which heads of 128 leave
  // room for: 267 us the chunk, 212 the trees.)
  static constexpr bool kTurns = R < 64;
  static constexpr int kGroups = kTurns ? 2 : 4, kCols = kTurns ? R : R / kGroups;  // a group's rows of a tile
  // the warps: softmax, copies, issuers of S and of P V, look-ups and scales, the walk
  static constexpr int kSoft = 4 * kGroups, kMmaS = kSoft + kC8Prod, kMmaO = kMmaS + 1, kLook = kMmaO + 1, kWalk = kLook + 1;
  static constexpr int kThreads = 32 * (kWalk + 1), kReaders = kWalk;  // (all but the walk take its parts)
  static constexpr int kOs = kTurns ? 2 : 1, kMix = kTurns ? 3 * R : 1;
  static constexpr uint32_t kQBox = kN * 128, kBox = kC8T * 128, kSlot = kC8T * HD;
  static constexpr int kSlots = HD == 128 ? (R < 64 ? 10 : 9) : R < 64 ? 5 : 4;
  static constexpr int kS = R < 64 ? 4 : HD == 256 ? 2 : 3;  // S buffers
  // Registers of the softmax's threads and of the others, of kRegs a thread at the launch:
  // 32 rows a thread do not fit 128, nor 16 of them 80, and every spilled value would queue
  // behind the copies.
  static constexpr int kRegs = kThreads == 512 ? 128 : 80;
  static constexpr int kSoftRegs = R < 32 ? kRegs : R == 32 ? 168 : 96, kOtherRegs = R < 32 ? kRegs : R == 32 ? 88 : 48;
  static_assert(32 * (kSoft * kSoftRegs + 8 * kOtherRegs) <= kThreads * kRegs, "registers of the launch");
  // P V's barriers: as many tiles as the look-ups may lead by.  The pages and scales of twice
  // as many are held.
  static constexpr uint32_t kPv = HD == 128 ? 8 : 4, kAhead = 2 * kPv;
  static constexpr uint32_t kQBytes = (kHalves * kQBox + 1023) / 1024 * 1024;
  // P's two buffers are boxes of a token a row, with its hi and mid terms and, up to 32 rows, lo;
  // of 64 rows the lo terms of both buffers fill a third box.
  static constexpr uint32_t kPOff = kQBytes, kLoBox = kPOff + 2 * kBox, kRingOff = kLoBox + (R < 64 ? 0 : kBox);
  static constexpr uint32_t kCtrlOff = kRingOff + kSlots * kSlot;
  // O has columns for each of P's terms (and zeros, of 8 rows, to a multiple of 16) where TMEM has
  // room for them; else a second MMA adds V lo to mid's.  (Two MMAs of 8 rows: decode of 16
  // sequences 103.2 us for 102.9, 600 rows over 200 to 800 tokens 69.0 for 68.3.)
  static constexpr bool kThree = R < 32;
  static constexpr int kON = kThree ? (3 * R + 15) / 16 * 16 : kN;
  static constexpr uint32_t kOCols = kHalves * kON, kSCol = kOs * kOCols;  // TMEM: O's halves, then S
  static_assert(kSCol + kS * kN <= 512, "TMEM has 512 columns");
  // kind::f8f6f4, D f32, A and B e4m3, M = 128, N = kN; O: A and B MN-major, B e5m2
  static constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kN >> 3) << 17) | ((128u >> 4) << 24);
  static constexpr uint32_t kIdescO =
      (1u << 4) | ((uint32_t)(kON >> 3) << 17) | ((128u >> 4) << 24) | (1u << 10) | (1u << 15) | (1u << 16);
  static constexpr uint32_t kIdescLo = kIdescO - ((uint32_t)((kON - R) >> 3) << 17);
};

// What beginning a unit costs, in tiles: its Q, its first references and its output.  At 3, 6, 9
// and 13 tiles (with weights of two terms), single rows of 32 heads over 8 over 300 to 9001 tokens
// took 42.5, 44.3, 47.2 and 46.4 us, and 64 single rows over 100 to 2000 tokens 24.8, 25.7, 27.3
// and 27.9; trees of 5 to 37 rows of 16 heads over 2 (units of 64 rows) 109, 106, 99 and 108.
template <int R>
constexpr int c8_start() { return R < 64 ? 3 : 9; }

struct C8Seq {
  SeqView v;
  int32_t tiles, m_tiles;  // in every unit's list; units of rows
  int64_t count;           // tiles of all its units, their starts included, a team's counted once
};

// How the launch shares its work out.
struct C8Plan {
  FastDiv group_div;
  int32_t head_log;  // log2 of the CTAs of a team, which take the same tiles of as many KV heads
  int32_t span;      // rows of a sequence that a unit holds of, at most
};

// Tiles that hold the first tokens (all of them where there is no window).
__device__ __forceinline__ int32_t first_tiles(const Cache8Args &a, const SeqView &v) {
  return (min(a.n_first, v.ctx + v.rows) + kC8T - 1) / kC8T;
}

// The units' lists have one length: that of the longest where a window cuts them.
template <int R>
__device__ __forceinline__ C8Seq c8_seq(const Cache8Args &a, const C8Plan &p, const SeqRaw &raw) {
  constexpr int kLog = R == 8 ? 3 : R == 16 ? 4 : R == 32 ? 5 : 6;
  static_assert(1 << kLog == R, "rows of a unit");
  C8Seq q;
  q.v = view_seq(a.seqs, raw);
  q.tiles = q.v.rows > 0 ? (q.v.ctx + q.v.rows + kC8T - 1) / kC8T : 0;
  if (a.window > 0 && q.tiles > 0) {
    const int64_t span = (int64_t)a.window + (a.seqs.mask ? q.v.rows : p.span);
    q.tiles = (int32_t)min((int64_t)q.tiles, first_tiles(a, q.v) + (span + kC8T - 1) / kC8T + 1);
  }
  q.m_tiles = (int32_t)(((int64_t)q.v.rows * a.group + R - 1) >> kLog);
  q.count = q.tiles > 0 ? (int64_t)(q.tiles + c8_start<R>()) * q.m_tiles * (a.nkv >> p.head_log) : 0;
  return q;
}

// One CTA's part of one unit.
struct C8Seg {
  int32_t s, kvh, m0;         // sequence, KV head, this CTA's unit's first row
  int32_t n;                  // tiles to process
  int32_t first, gap, near;   // tile i of the part is token tile first + i, gap less from `near` on
  int32_t back;               // no row sees the tokens from n_first to before `back`
  int32_t row0, rows, ctx;    // the sequence's
  int32_t flags;
  enum : int32_t {
    kWhole = 1,  // the unit's every tile
    kHead = 2,   // the unit began in an earlier CTA
    kEmpty = 4,  // none of its tiles (a share that ends in a unit's start), or no rows
    kEnd = 8     // no part: the walk is over
  };
  __device__ int32_t tile(int i) const { return first + i - (i >= near ? gap : 0); }
  // whether token t may be seen by a row (others are not read)
  __device__ bool wants(const Cache8Args &a, int32_t t) const { return t < ctx + rows && (t < a.n_first || t >= back); }
};

// The unit whose first tiles a CTA ends with, and the team that has its last ones; -1: none.
struct C8Open {
  int32_t row0, rows, m0, kvh, last;
};

// Walks a team's share of the list, unit by unit, the sequences' lengths read one ahead.
template <int R>
struct C8Walk {
  const Cache8Args &a;
  const C8Plan &p;
  int64_t left, off;
  int32_t s;
  C8Seq q;
  SeqRaw ahead;
  int32_t rest;  // of the unit whose part next() gave, the tiles behind it
  __device__ C8Walk(const Cache8Args &a_, const C8Plan &p_, int32_t s_, int64_t off_, int64_t left_)
      : a(a_), p(p_), left(left_), off(off_), s(s_) {
    if (left <= 0) return;
    q = c8_seq<R>(a, p, read_seq(a.seqs, s));
    ahead = read_seq(a.seqs, min(s + 1, a.seqs.n_seqs - 1));
  }
  __device__ C8Seg next() {
    C8Seg g = {};
    g.flags = C8Seg::kEnd;
    if (left <= 0) return g;
    while (off >= q.count) {
      off -= q.count;
      if (++s >= a.seqs.n_seqs) {
        left = 0;
        return g;
      }
      q = c8_seq<R>(a, p, ahead);
      ahead = read_seq(a.seqs, min(s + 1, a.seqs.n_seqs - 1));
    }
    const int32_t length = q.tiles + c8_start<R>();
    int32_t unit;  // (team of KV heads, rows)
    if ((off >> 31) == 0) unit = (int32_t)((uint32_t)off / (uint32_t)length);
    else unit = (int32_t)(off / length);
    const int32_t from = (int32_t)(off - (int64_t)unit * length);
    const int32_t part = (int32_t)min((int64_t)(length - from), left);
    off += part;
    left -= part;
    const int32_t i0 = max(0, from - c8_start<R>()), take = max(0, from + part - c8_start<R>()) - i0;
    rest = q.tiles - i0 - take;
    g.s = s;
    const int32_t heads = unit / q.m_tiles, mt = unit - heads * q.m_tiles;
    g.kvh = (heads << p.head_log) + ((int32_t)blockIdx.x & ((1 << p.head_log) - 1));
    g.row0 = q.v.row0;
    g.rows = q.v.rows;
    g.ctx = q.v.ctx;
    g.first = i0;
    const int64_t m0 = (int64_t)mt * R, m_all = (int64_t)q.v.rows * a.group;
    g.flags = (take == q.tiles ? C8Seg::kWhole : 0) | (i0 > 0 ? C8Seg::kHead : 0);
    if (take == 0 || m0 >= m_all) {
      g.flags |= C8Seg::kEmpty;
      return g;
    }
    // the token tiles that this unit's rows see any of: those of the first tokens, and from
    // `back` (its first row's oldest) to `end` (its last row's newest)
    g.m0 = (int32_t)m0;
    const bool chain = a.seqs.mask == nullptr;
    const int32_t j0 = fast_div(p.group_div, (int32_t)m0), j1 = fast_div(p.group_div, (int32_t)(min(m0 + R, m_all) - 1));
    const int32_t end = (q.v.ctx + (chain ? j1 + 1 : q.v.rows) + kC8T - 1) / kC8T;
    int32_t count = end;
    g.near = 0x7FFFFFFF;
    if (a.window > 0) {
      // Where they leave tiles out between them, the window's come first: a reference is to
      // be taken from a tile that the rows see much of.
      g.back = max(0, q.v.ctx + (chain ? j0 : 0) - (a.window - 1));
      const int32_t near = min(end, first_tiles(a, q.v)), from_back = min(g.back / kC8T, end);
      if (from_back > near) {
        count = end - from_back + near;
        g.first = i0 + from_back;
        g.near = max(0, end - from_back - i0);
        g.gap = end;
      }
    }
    g.n = max(0, min(take, count - i0));
    return g;
  }
};

template <int kMix, int kAhead>
struct C8Ctrl {
  float factor[kC8MostRows];    // log2 units a unit of S and ks
  float less_ref[kC8MostRows];  // [group][its rows]: the reference, negated
  // [group][its rows]: what a move multiplies by.  A part's output has 1 / sum there where
  // a group writes out its own rows: its warps meet before the next move.
  float alpha[kC8MostRows];
  float mix[kMix];  // else, [2][row]: the groups' join at a part's end, and [2R + row]: 1 / sum
  int64_t where[kC8MostRows];   // a row's place in the output
  int32_t depth[kC8MostRows];
  C8Seg segs[kC8Segs];
  // [tile % kAhead][16 tokens]: the pool's row of the first that is read (-1: none), scales
  int32_t slots[kAhead][8];
  float scales[kAhead][2][8];
  uint64_t full[10], empty[10], looked[kAhead], scaled[kAhead];
  uint64_t s_full[4], s_free[4], p_ready[2], pv_done[kAhead / 2];
  uint64_t q_full, o_free, drain[2], seg_full[kC8Segs], seg_free[kC8Segs];
  int32_t bad[2], abort;
  uint32_t tmem_base;
};
template <int kMix, int kAhead>
union C8Scratch {  // the plan is made before anything else
  C8Ctrl<kMix, kAhead> c;
  ShareScratch share;
};
template <int HD, int R>
constexpr size_t c8_smem() { return C8Geom<HD, R>::kCtrlOff + sizeof(C8Scratch<C8Geom<HD, R>::kMix, C8Geom<HD, R>::kAhead>); }
static_assert(c8_smem<256, 64>() <= 232448 && c8_smem<128, 64>() <= 232448, "227 KiB per CTA");

// Ring position of tile j's V among a part's n tiles, counted from the part's first copy:
// K0, K1, V0, K2, V1, ..., V(n-1), about the order the MMAs take them in.
__device__ __forceinline__ int c8_v_pos(int j, int n) { return j + 1 < n ? 2 + 2 * j : 2 * n - 1; }

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Bounded wait on a phase.  Every role's loop has several and they share the instruction
// cache, so it is short: after a test, a look at the abort flag and the clock and one
// instruction that sleeps until the phase completes or some time has passed.
__device__ __forceinline__ bool phase_done(uint32_t mb, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(mb), "r"(parity), "r"(kC8SuspendNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool one_wait(uint32_t mb, uint32_t parity, long long limit, volatile int32_t *abort_flag) {
  if (mbar_test(mb, parity)) return true;
  const long long t0 = clock64();
  do {
    if (*abort_flag) return false;
    if (clock64() - t0 > limit) {
      *abort_flag = 1;
      return false;
    }
  } while (!phase_done(mb, parity));
  return true;
}
// ... of a warp, each lane for itself, the verdict the warp's.
__device__ __forceinline__ bool warp_wait(uint32_t mb, uint32_t parity, long long limit, volatile int32_t *abort_flag) {
  return __all_sync(0xffffffffu, one_wait(mb, parity, limit, abort_flag));
}

// 4 bytes from global to shared memory, asynchronously; bytes 0: zeros.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// D += A B of 8-bit types.
__device__ __forceinline__ void mma_8(uint32_t dtmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
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

// A column of O's halves (`half` columns apart) and its other terms (`term` columns on), times `by`.
template <int kHalves, int kTerms>
__device__ __forceinline__ void tmem_scale(uint32_t taddr, uint32_t half, uint32_t term, float by) {
  uint32_t x[kTerms * kHalves];
#pragma unroll
  for (int i = 0; i < kTerms * kHalves; ++i)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x[i]) : "r"(taddr + (i / kTerms) * half + (i % kTerms) * term));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < kTerms * kHalves; ++i) {
    asm volatile("" : "+r"(x[i])::"memory");
    x[i] = __float_as_uint(__uint_as_float(x[i]) * by);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr + (i / kTerms) * half + (i % kTerms) * term), "r"(x[i])
                 : "memory");
  }
}

__device__ __forceinline__ void tmem_scale1(uint32_t taddr, float by) {
  uint32_t x;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(x)::"memory");
  x = __float_as_uint(__uint_as_float(x) * by);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(x) : "memory");
}

// 1 / x within 2^-23 of it, and log2 x (within 2^-22, or 2^-22 of it outside [1/2, 2]): short,
// for code that runs once a part.
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ref + log2 of a sum, in units of e: x = 2^e m (a normal number) with m in [3/4, 3/2), whose
// logarithm is within 2^-22.  A sum that is not finite is the result: taken apart, its bits
// would give a number.
__device__ __forceinline__ float lse_of(float ref, float x) {
  if (!(x < INFINITY)) return x;
  const int32_t e = ((int32_t)__float_as_uint(x) - 0x3F400000) >> 23;
  const float m = __uint_as_float(__float_as_uint(x) - ((uint32_t)e << 23));
  return (ref + (float)e + lg2(m)) * 0.6931471805599453f;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// K values of each lane joined over the lanes: lane i gets the K-th of value i / (32 / K).
// Half of the values change lanes in each step, so that all are joined at once.
template <int K, typename Join>
__device__ __forceinline__ float over_lanes(float (&x)[K], int lane, Join &&join) {
  int o = 16;
#pragma unroll
  for (int half = K / 2; half > 0; half /= 2, o /= 2) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? x[i + half] : x[i], give = upper ? x[i] : x[i + half];
      x[i] = join(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
#pragma unroll
  for (int p = 16 / K; p > 0; p /= 2) x[0] = join(x[0], __shfl_xor_sync(0xffffffffu, x[0], p));
  return x[0];
}

// Two values as e4m3 terms hi + lo / 16: exact for eight bits, as bf16 has, of 2^-6 and more.
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

// Two values of 0 to 57344 as e5m2 terms hi + (mid + lo) / 4, the upper bytes of f16 halves: an
// e5m2 is an f16's upper byte, so hi and mid are cut off by a mask (a NaN's stays one) and lo is
// rounded by adding half a step.  hi leaves eight of an f16's eleven bits, at most 8160, mid five,
// of which lo has three: off by 2^-9 of a value, by 2^-11 for its f16, or by 2^-19.
__device__ __forceinline__ void split_e5m2(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
  asm("{\n\t.reg .b32 t, s;\n\tsub.f16x2 t, %1, %2;\n\tmov.b32 s, 0x44004400;\n\tmul.f16x2 %0, t, s;\n\t}"  // 4
      : "=r"(mid)
      : "r"(hi), "r"(hi & 0xFF00FF00u));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(mid), "r"(mid & 0xFF00FF00u));
  lo += 0x00800080u;
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
// ... over all groups (`threads` of them)
__device__ __forceinline__ void soft_sync(int threads) { asm volatile("barrier.cta.sync 5, %0;" ::"r"(threads) : "memory"); }
__device__ __forceinline__ bool soft_any(int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, 5, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int g) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + g) : "memory"); }

__device__ __forceinline__ bool nan8(uint32_t byte) { return (byte & 0x7Fu) == 0x7Fu; }

template <int HD, int R>
__global__ void __launch_bounds__(C8Geom<HD, R>::kThreads, 1)
cache8_attn_kernel(const Cache8Args a, const C8Plan plan, C8Open *__restrict__ open, float2 *__restrict__ part_ml, float *__restrict__ part_o) {
  using G = C8Geom<HD, R>;
  extern __shared__ __align__(1024) uint8_t c8_shared[];
  auto &both = *reinterpret_cast<C8Scratch<G::kMix, G::kAhead> *>(c8_shared + G::kCtrlOff);
  auto &C = both.c;
  const uint32_t sQ = sm32(c8_shared), sP = sm32(c8_shared + G::kPOff), sRing = sm32(c8_shared + G::kRingOff);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const long long lim = a.wait_limit > 0 ? a.wait_limit : kC8SpinLimit;
  volatile int32_t *abort_flag = &C.abort;

  grid_dependency_sync();  // before TMEM too: an earlier launch may hold it
  // ---- the plan
  const uint32_t teams = gridDim.x >> plan.head_log, my_team = blockIdx.x >> plan.head_log;
  const FoundShare found = find_share(a.seqs.n_seqs, G::kThreads, teams, my_team, both.share, [&](int32_t s) -> int64_t {
    if (s >= a.seqs.n_seqs) return 0;
    const C8Seq q = c8_seq<R>(a, plan, read_seq(a.seqs, s));
    if (!q.v.ok && blockIdx.x == 0) report_error(a.status, kErrRowRange, s);
    return q.count;
  });
  __syncthreads();  // the plan's scratch lies where the barriers do
  if (tid == 0) {
    for (int i = 0; i < G::kSlots; ++i) {
      mbar_init(sm32(&C.full[i]), 32 * kC8Prod);
      mbar_init(sm32(&C.empty[i]), 1);
    }
    for (int i = 0; i < (int)G::kPv; ++i) mbar_init(sm32(&C.pv_done[i]), 1);
    for (int i = 0; i < (int)G::kAhead; ++i) {
      mbar_init(sm32(&C.looked[i]), 8);
      mbar_init(sm32(&C.scaled[i]), 8);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(sm32(&C.s_full[b]), 2);
      mbar_init(sm32(&C.s_free[b]), G::kSoft / G::kOs);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sm32(&C.p_ready[b]), G::kSoft / G::kOs);
      mbar_init(sm32(&C.drain[b]), 1);
      C.bad[b] = 0;
    }
    for (int i = 0; i < kC8Segs; ++i) {
      mbar_init(sm32(&C.seg_full[i]), 1);
      mbar_init(sm32(&C.seg_free[i]), G::kReaders);
    }
    mbar_init(sm32(&C.q_full), G::kSoft);
    mbar_init(sm32(&C.o_free), G::kSoft);
    C.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == G::kMmaS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm32(&C.tmem_base)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem_base;
  const bool laid_out = (sQ & 1023u) == 0;  // the swizzle needs it; the declaration asks for it
  // A warp's next part.  False where the wait for it gave up.
  uint32_t segs_taken = 0;
  auto take_seg = [&](C8Seg &g) -> bool {
    const uint32_t i = segs_taken % kC8Segs;
    const bool ok = warp_wait(sm32(&C.seg_full[i]), (segs_taken / kC8Segs) & 1u, lim, abort_flag);
    __syncwarp();
    if (ok) g = C.segs[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(sm32(&C.seg_free[i]));
    ++segs_taken;
    return ok;
  };

  if (warp >= G::kSoft && warp < G::kMmaS) {
    if constexpr (G::kOtherRegs < G::kRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kOtherRegs));
    C8Seg g;
    // ---- producers: warp p brings 32 of a tile's tokens, 512 bytes an instruction (kRows
    // rows).  A block's tokens, and so 16 of a tile's from a multiple of 16 on, lie in one
    // page: two places a tile.  A slot's barrier takes each thread's arrival when its copies
    // have landed, so the whole ring may be in flight.
    constexpr int kCh = HD / 16, kRows = 32 / kCh, kN = 16 / kRows;  // chunks of a row, copies of 16 tokens
    const int p0 = (warp - G::kSoft) * 32, ch = lane % kCh, hl = lane / kCh;
    const uint32_t dst0 = sRing + (uint32_t)(ch >> 3) * G::kBox + (uint32_t)(p0 + hl) * 128u;
    const int64_t pitch = (int64_t)a.nkv * HD;
    const int64_t step = kRows * pitch;
    uint32_t slot = 0u, phase = 0u, jg = 0u;
    bool ok = true;
    while (ok && take_seg(g) && !(g.flags & C8Seg::kEnd)) {
      const int32_t kv = g.ctx + g.rows;
      const int64_t mine = (int64_t)g.kvh * HD + ch * 16 + hl * pitch;
      // copies in the ring's order: K0, K1, V0, K2, V1, ..., V(n - 1)
      int j = 0;         // the tile of this copy
      bool is_k = true;
      for (int i = 0; i < 2 * g.n; ++i) {
        const uint32_t at = (jg + (uint32_t)j) % G::kAhead;
        if (!warp_wait(sm32(&C.looked[at]), ((jg + (uint32_t)j) / G::kAhead) & 1u, lim, abort_flag) ||
            !warp_wait(sm32(&C.empty[slot]), phase ^ 1u, lim, abort_flag)) {
          ok = false;
          break;
        }
        const uint8_t *const pool = is_k ? a.k_pool : a.v_pool;
        const int32_t t0 = g.tile(j) * kC8T + p0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int32_t first = C.slots[at][p0 / 16 + e], t = t0 + 16 * e;
          const uint32_t dst = dst0 + slot * G::kSlot + (uint32_t)e * 16u * 128u;
          // row p0 + 16 e + kRows k + hl, its 16-byte chunks swizzled by row % 8
          auto to = [&](int k) { return dst + (uint32_t)(k * kRows) * 128u + (uint32_t)(((ch & 7) ^ ((kRows * k + hl) & 7)) << 4); };
          if (first >= 0 && t + 16 <= kv && (t + 16 <= a.n_first || t >= g.back)) {  // all of them
            const uint8_t *src = pool + (int64_t)first * pitch + mine;
#pragma unroll
            for (int k = 0; k < kN; ++k) {
              cp_async16(to(k), src, 16u);
              src += step;
            }
          } else {
            // `first` is that of token t, or of the first one that the window leaves
            const int64_t skip = g.wants(a, t) ? 0 : g.back - t;
#pragma unroll 1
            for (int k = 0; k < kN; ++k) {
              const bool read = first >= 0 && g.wants(a, t + kRows * k + hl);
              cp_async16(to(k), read ? pool + (first - skip) * pitch + mine + k * step : pool, read ? 16u : 0u);
            }
          }
        }
        cp_async_arrive(sm32(&C.full[slot]));
        if (++slot == (uint32_t)G::kSlots) {
          slot = 0u;
          phase ^= 1u;
        }
        // K of tile j is followed by V of tile j - 1 (K0 by K1, where there is one), V of
        // tile j by K of tile j + 2, and the last ones by V
        if (is_k) {
          if (j == 0 && g.n > 1) {
            j = 1;
          } else {
            is_k = false;
            j = max(0, j - 1);
          }
        } else if (j + 2 < g.n) {
          is_k = true;
          j += 2;
        } else {
          ++j;
        }
      }
      jg += (uint32_t)g.n;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives the CTA
  } else if (warp >= G::kMmaS) {
    if constexpr (G::kOtherRegs < G::kRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kOtherRegs));
    if (warp == G::kWalk) {
      // ---- the walk
      C8Walk<R> walk(a, plan, found.seq, found.off, laid_out ? found.share.n : 0);
      C8Open last = {0, 0, 0, 0, -1};
      for (uint32_t k = 0;; ++k) {
        const C8Seg g = walk.next();
        if (!(g.flags & (C8Seg::kEnd | C8Seg::kEmpty | C8Seg::kHead | C8Seg::kWhole)))  // (then the share ends here)
          last = {g.row0, g.rows, g.m0, g.kvh, (int32_t)(my_team + (walk.rest + found.share.per - 1) / found.share.per)};
        if (k >= kC8Segs && !warp_wait(sm32(&C.seg_free[k % kC8Segs]), ((k / kC8Segs) & 1u) ^ 1u, lim, abort_flag)) break;
        __syncwarp();
        if (lane == 0) {
          C.segs[k % kC8Segs] = g;
          mbar_arrive(sm32(&C.seg_full[k % kC8Segs]));
        }
        if (g.flags & C8Seg::kEnd) break;
      }
      if (lane == 0) open[blockIdx.x] = last;
    } else if (warp == G::kLook) {
      // ---- the look-ups: lane 8 i + e takes 16 tokens of the i-th of four tiles.  Under load
      // a read takes several thousand cycles, so the pages of the next four tiles are read
      // ahead.  Four tiles take the places of those kAhead before them once P V of the tile kPv
      // before the first of them is done.
      const int ti = lane >> 3, e = lane & 7;
      uint32_t jg = 0;
      bool ok = true;
      C8Seg g;
      while (ok && take_seg(g) && !(g.flags & C8Seg::kEnd)) {
        const int32_t kv = g.ctx + g.rows;
        // the first token that is read of this lane's 16 of tile j, -1: none
        auto token = [&](int j) -> int32_t {
          if (j >= g.n) return -1;
          const int32_t t = g.tile(j) * kC8T + 16 * e;
          if (g.wants(a, t)) return t;
          return t < kv && t + 16 > g.back && g.back < kv ? g.back : -1;
        };
        auto page_of = [&](int32_t t) -> int32_t {
          return t < 0 ? 0 : a.seqs.table[(int64_t)g.s * a.seqs.table_cols + fast_div(a.seqs.page, t)];
        };
        int32_t t = token(ti), page = page_of(t);
        for (int j = 0; j < g.n; j += 4) {
          const int32_t t_next = token(j + 4 + ti), page_next = page_of(t_next);
          const int count = min(4, g.n - j);
          const uint32_t at = (jg + (uint32_t)ti) % G::kAhead;
          // (P V of tile jg cannot have been done, and that of tile jg - 2 kPv has been waited for)
          if (jg >= G::kPv && !warp_wait(sm32(&C.pv_done[jg % G::kPv]), ((jg / G::kPv) & 1u) ^ 1u, lim, abort_flag)) {
            ok = false;
            break;
          }
          if (ti < count) {
            const bool there = t >= 0 && (uint32_t)page < (uint32_t)a.seqs.pool_pages;
            if (t >= 0 && !there) report_error(a.status, kErrTokenRange, g.s);
            const int32_t slot = there ? page * a.seqs.page.d + (t - fast_div(a.seqs.page, t) * a.seqs.page.d) : -1;
            C.slots[at][e] = slot;
            mbar_arrive(sm32(&C.looked[at]));
            const int64_t block = there ? (int64_t)(slot >> a.unit_log) * a.nkv + g.kvh : 0;
            cp_async4(sm32(&C.scales[at][0][e]), a.k_scale + block, there ? 4u : 0u);
            cp_async4(sm32(&C.scales[at][1][e]), a.v_scale + block, there ? 4u : 0u);
            cp_async_arrive(sm32(&C.scaled[at]));
          }
          jg += (uint32_t)count;
          t = t_next;
          page = page_next;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    // ---- MMA issuers: the warp steps through its tiles, one elected lane issues
    if (warp <= G::kMmaO) {
      C8Seg g;
      bool ok = true;
      auto wait = [&](uint64_t &bar, uint32_t parity) {
        ok = ok && warp_wait(sm32(&bar), parity, lim, abort_flag);
        return ok;
      };
      auto take_one = [&]() -> bool {
        if (!take_seg(g)) return false;
        g.n = __shfl_sync(0xffffffffu, g.n, 0);
        return !(g.flags & C8Seg::kEnd);
      };
      const bool lead = elect_one();
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
      // tile whose S this warp issued, or V of tile j - 4 or an earlier one, whose P V
      // was waited for, or, in a part's first tiles, of an earlier part, all of whose P V
      // were done before this part's Q was stored.  P V of tile j: it is V, or K of an
      // earlier tile.
      auto landed = [&]() {
        if (!wait(C.full[slot], phase)) return false;
        // the copies wrote through the generic proxy; the MMAs read through the async one
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_after();
        return true;
      };
      const uint32_t desc_hi = (uint32_t)(sw128_desc(0) >> 32);
      uint32_t jg = 0, part = 0;  // tiles and parts before this one
      if (warp == G::kMmaS) {
        const uint32_t q_lo = (uint32_t)sw128_desc(sQ), r_lo = (uint32_t)sw128_desc(sRing);
        uint32_t b = 0, b_phase = 1;  // S buffer, parity of its s_free phase before this use
        while (ok && take_one()) {
          if (g.n == 0) continue;
          if (!wait(C.q_full, part & 1u)) break;
          ++part;
          for (int j = 0; j < g.n; ++j, ++jg) {
            if (jg >= (uint32_t)G::kS && !wait(C.s_free[b], b_phase)) break;  // tile j - kS is read
            if (jg >= 4 && !wait(C.pv_done[(jg - 4u) % G::kPv], ((jg - 4u) / G::kPv) & 1u)) break;
            if (j > 0) step(j == 1 ? 1u : 2u);
            // (the tile's scales: one wait less for the many)
            if (!wait(C.scaled[jg % G::kAhead], (jg / G::kAhead) & 1u) || !landed()) break;
            const uint32_t d = tmem + G::kSCol + b * G::kN, k_lo = r_lo + slot * (G::kSlot >> 4);
            if (lead) {
#pragma unroll
              for (int kk = 0; kk < HD / 32; ++kk) {
                const uint32_t in = (uint32_t)(kk & 3) * 2u;  // 32 bytes
                mma_8(d, desc_of(k_lo + (uint32_t)(kk >> 2) * (G::kBox >> 4) + in, desc_hi),
                         desc_of(q_lo + (uint32_t)(kk >> 2) * (G::kQBox >> 4) + in, desc_hi), G::kIdescS, kk > 0 ? 1u : 0u);
              }
              mma_commit(sm32(&C.empty[slot]));
              mma_commit(sm32(&C.s_full[b]));
              mbar_arrive(sm32(&C.s_full[b]));
            }
            __syncwarp();
            if (++b == (uint32_t)G::kS) {
              b = 0;
              b_phase ^= 1u;
            }
          }
          step(g.n == 1 ? 2u : 3u);  // past V(n - 2) and V(n - 1)
        }
      } else {
        const uint32_t r_lo = (uint32_t)sw128_mn_desc(sRing, 0), p_lo = (uint32_t)sw128_mn_desc(sP, 0);
        // the lo terms' place beside p, and from one buffer to the next
        constexpr uint32_t kLoAt = R < 64 ? 2 * R : 2 * G::kBox, kLoStep = R < 64 ? G::kBox : 64u;
        while (ok && take_one()) {
          if (g.n == 0) continue;
          if (part > 0 && !wait(C.o_free, (part - 1) & 1u)) break;  // the part before has left O
          ++part;
          for (int j = 0; j < g.n; ++j, ++jg) {
            if (!wait(C.p_ready[jg & 1u], (jg >> 1) & 1u)) break;
            step(j + 1 < g.n ? 2u : 1u);
            if (!landed()) break;
            const uint32_t o = tmem + (G::kTurns ? (jg & 1u) * G::kOCols : 0u);
            const uint32_t p = p_lo + (jg & 1u) * (G::kBox >> 4), p3 = p_lo + (kLoAt >> 4) + (jg & 1u) * (kLoStep >> 4);
            const uint32_t v_lo = r_lo + slot * (G::kSlot >> 4);
            if (lead) {
#pragma unroll
              for (int h = 0; h < G::kHalves; ++h)
#pragma unroll
                for (int kk = 0; kk < kC8T / 32; ++kk) {  // 32 tokens a step: 4 KiB of V's and of P's rows
                  const uint64_t v = desc_of(v_lo + (uint32_t)h * (G::kBox >> 4) + 256u * kk, desc_hi);
                  const uint32_t d = o + (uint32_t)h * G::kON;
                  mma_8(d, v, desc_of(p + 256u * kk, desc_hi), G::kIdescO, (j >= G::kOs || kk > 0) ? 1u : 0u);
                  if constexpr (!G::kThree) mma_8(d + R, v, desc_of(p3 + 256u * kk, desc_hi), G::kIdescLo, 1u);
                }
              mma_commit(sm32(&C.empty[slot]));
              mma_commit(sm32(&C.pv_done[jg % G::kPv]));
            }
            __syncwarp();
          }
          step(1u);
        }
      }
      // every MMA this warp issued has finished before TMEM is freed
      if (lead) mma_commit(sm32(&C.drain[warp - G::kMmaS]));
      __syncwarp();
      if (lane == 0) tc_wait(sm32(&C.drain[warp - G::kMmaS]), 0u, kC8SpinLimit, nullptr);
    }
    __syncwarp();
  } else {
    if constexpr (G::kSoftRegs > G::kRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kSoftRegs));
    // ---- softmax: thread tk has the tile's token tk (TMEM lane) and, at the end, dims tk
    // and tk + 128.  Group w takes every other tile, or its rows of each.  After an abort
    // every wait returns at once, and the loops and barriers run on to the end.
    constexpr int kCols = G::kCols;
    const int w = warp >> 2, wq = warp & 3, tk = wq * 32 + lane;
    const int n0 = G::kTurns ? 0 : w * kCols;  // this group's first row
    float *const less_ref = C.less_ref + w * kCols, *const alpha = C.alpha + w * kCols;
    float *const inverse = G::kTurns ? C.mix + 2 * R : C.alpha;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t my_o = lane_base + (G::kTurns ? w * G::kOCols : (uint32_t)n0);
    // P V of tile i.  A warp has waited for tile i - 4 (or a later one) by then, so of a
    // barrier no phase but the last two is ever in question.
    auto wait_pv = [&](uint32_t i) { warp_wait(sm32(&C.pv_done[i % G::kPv]), (i / G::kPv) & 1u, lim, abort_flag); };
    // This warp's rows of a part's Q, split into two e4m3 terms, with what goes with a row.
    constexpr int kLanes = HD / 8, kPer = 32 / kLanes;  // lanes a row, rows a warp takes at once
    constexpr int kTimes = (R + G::kSoft * kPer - 1) / (G::kSoft * kPer);
    static_assert(kTimes <= 4, "rows of Q held in registers between their fetch and their split");
    const int ch = lane % kLanes, sub = lane / kLanes;
    auto row_of = [&](int i) { return (i * G::kSoft + warp) * kPer + sub; };
    uint4 raw[kTimes];
    auto fetch_q = [&](const C8Seg &e) {
#pragma unroll
      for (int i = 0; i < kTimes; ++i) {
        const int n = row_of(i);
        const bool valid = n < R && e.m0 + n < e.rows * a.group;
        const int32_t m = valid ? e.m0 + n : 0, j = fast_div(plan.group_div, m);
        const int32_t head = e.kvh * a.group + (m - j * a.group);
        raw[i] = valid ? ldg_v4(a.q + (int64_t)(e.row0 + j) * a.q_stride + (int64_t)head * HD + 8 * ch) : make_uint4(0, 0, 0, 0);
      }
    };
    auto store_q = [&](const C8Seg &e) {
      const int32_t m_all = e.rows * a.group;
#pragma unroll
      for (int i = 0; i < kTimes; ++i) {
        const int n = row_of(i);
        const bool mine = n < R, valid = mine && e.m0 + n < m_all;
        // the largest magnitude; of a row with one that is not finite, that one, and NaN below
        uint32_t top = __vmaxu2(__vmaxu2(raw[i].x & 0x7FFF7FFFu, raw[i].y & 0x7FFF7FFFu),
                                __vmaxu2(raw[i].z & 0x7FFF7FFFu, raw[i].w & 0x7FFF7FFFu));
        top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // the least power of two s with it <= 448 s = 1.75 * 2^8 s, and 1 / s
        const int ex = max(-126, (int)(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0));
        const float s = __uint_as_float((uint32_t)(127 + ex) << 23), inv = __uint_as_float((uint32_t)(127 - ex) << 23);
        float x[8];
        unpack8(raw[i], x);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)  // (x + 0 x: an infinity becomes NaN, which the conversions keep)
          split_e4m3(fmaf(x[2 * k], 0.f, x[2 * k]) * inv, fmaf(x[2 * k + 1], 0.f, x[2 * k + 1]) * inv, hi[k], lo[k]);
        if (mine) {
          auto at = [&](int row) {  // 8 bytes of a 128-byte row of a box, its 16-byte chunks swizzled
            return c8_shared + (ch >> 4) * G::kQBox + row * 128 + (((ch >> 1) & 7) ^ (row & 7)) * 16 + (ch & 1) * 8;
          };
          *reinterpret_cast<uint2 *>(at(n)) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2 *>(at(R + n)) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          if (ch == 0) {
            C.factor[n] = a.scale_log2 * s;
#pragma unroll
            for (int o = 0; o < G::kOs; ++o) C.less_ref[o * kCols + n] = valid ? -kC8Unset : -kC8Nobody;
          }
        }
      }
      if (a.window > 0 && a.seqs.mask != nullptr) {  // the rows' drafted tokens, a lane a row
        for (int n = tid; n < R; n += 32 * G::kSoft) {
          int32_t depth = 0;
          if (e.m0 + n < m_all) {
            const uint32_t *mrow = a.seqs.mask + (int64_t)(e.row0 + fast_div(plan.group_div, e.m0 + n)) * a.seqs.mask_words;
            for (int32_t k = 0; 32 * k < e.rows; ++k) {
              const int32_t over = e.rows - 32 * k;
              depth += __popc(over >= 32 ? mrow[k] : mrow[k] & ((1u << over) - 1u));
            }
          }
          C.depth[n] = max(0, depth - 1);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(sm32(&C.q_full));
    };
    int32_t seg = 0;
    // Whether group o had a tile of part g, whose first went to group jg0 % 2.
    uint32_t jg = 0, ns = 0, loaded = 0, jg0 = 0;  // tiles, copies and parts with tiles before this one
    C8Seg g = {}, next;
    g.flags = C8Seg::kEmpty;
    auto has = [&](int o) { return G::kTurns ? g.n > (int)((jg0 + (uint32_t)o) & 1u) : g.n > 0; };
    auto write_out = [&]() {
      if (!(g.flags & C8Seg::kEmpty)) {
        const bool whole = (g.flags & C8Seg::kWhole) != 0;
        constexpr int kRows = R / G::kGroups, kOut = kRows < 8 ? kRows : 8;  // a group's rows of the output, at once
        const int first = w * kRows;
#pragma unroll 1
        for (int h = 0; h < G::kHalves; ++h) {
          const int d = h * 128 + tk;
#pragma unroll 1
          for (int c = first; c < first + kRows; c += kOut) {
            float x[kOut];
#pragma unroll
            for (int i = 0; i < kOut; ++i) x[i] = 0.f;
#pragma unroll
            for (int o = 0; o < G::kOs; ++o) {
              if (!has(o)) continue;
              uint32_t hi[kOut], mid[kOut], lo[kOut];
              const uint32_t at = lane_base + (uint32_t)o * G::kOCols + (uint32_t)(h * G::kON + c);
              tmem_cols<kOut>(at, hi);
              tmem_cols<kOut>(at + R, mid);
              if constexpr (G::kThree) tmem_cols<kOut>(at + 2 * R, lo);
              tmem_ready<kOut>(hi);
              tmem_ready<kOut>(mid);
              if constexpr (G::kThree) tmem_ready<kOut>(lo);
#pragma unroll
              for (int i = 0; i < kOut; ++i) {
                const float less = G::kThree ? __uint_as_float(mid[i]) + __uint_as_float(lo[i]) : __uint_as_float(mid[i]);
                const float y = fmaf(less, 0.25f, __uint_as_float(hi[i]));
                x[i] = G::kTurns ? fmaf(y, C.mix[o * kCols + c + i], x[i]) : y;
              }
            }
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
              const int64_t where = C.where[c + i];
              if (where < 0) continue;
              const float y = x[i] * inverse[c + i];
              if (whole) a.out[where + d] = (uint16_t)f32_to_bf16(y);
              else part_o[where + d] = y;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && g.n > 0) mbar_arrive(sm32(&C.o_free));
    };
    // the next part, unless a wait of one of the softmax's warps gave up
    auto advance = [&](C8Seg &to) -> bool {
      const bool ok = take_seg(to);
      return !soft_any(32 * G::kSoft, !ok) && !(to.flags & C8Seg::kEnd);
    };
    // Parts overlap: the next one's Q is fetched before this one's output is written.
    bool more = advance(next);
    if (more && next.n > 0) fetch_q(next);
    while (true) {
      if (more && next.n > 0) store_q(next);
      write_out();
      if (!more) break;
      g = next;
      ++seg;
      const int32_t m0 = g.m0, m_all = g.rows * a.group, kv = g.ctx + g.rows;
      const bool chain = a.seqs.mask == nullptr, empty = (g.flags & C8Seg::kEmpty) != 0;
      // whether a row may be blind to a token that another one sees, or that is read beside its own
      const bool veiled = g.rows > 1 || !chain || a.window > 0;
      const int32_t j0 = fast_div(plan.group_div, m0), j1 = fast_div(plan.group_div, max(0, min(m0 + R, m_all) - 1));
      // tokens below `clear` and, of a window, from `old` on or below n_first are seen by every row
      const int32_t clear = chain ? g.ctx + j0 + 1 : g.ctx;
      const int32_t old = a.window > 0 ? max(0, g.ctx + (chain ? j1 : g.rows - 1) - (a.window - 1)) : 0;
      const int32_t clear_tile = clear / kC8T, old_tile = (old + kC8T - 1) / kC8T, first_tile = a.n_first / kC8T;
      auto is_masked = [&](int32_t tile) { return tile >= clear_tile || (tile < old_tile && tile >= first_tile); };
      // the columns of rows [from, to) of the sequence, among this group's
      auto columns = [&](int32_t from, int32_t to) -> uint32_t {
        const int lo = min(max(from * a.group - m0 - n0, 0), kCols), hi = min(max(to * a.group - m0 - n0, 0), kCols);
        if (lo >= hi) return 0u;
        return (hi >= 32 ? 0xFFFFFFFFu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
      };
      // which of this group's rows see token t
      auto sees = [&](int32_t t) -> uint32_t {
        if (t >= kv) return 0u;
        const int32_t k = t - g.ctx;
        if (chain) {  // row j: k <= j, and j - k < window or t < n_first
          // (k + window may pass 31 bits, where the table's end is near them; rows - k does not)
          const bool near = a.window > 0 && t >= a.n_first && g.rows - k > a.window;
          return columns(max(k, 0), near ? max(0, k + a.window) : g.rows);
        }
        uint32_t s = 0u;
        if (k >= 0) {
          const int32_t end = fast_div(plan.group_div, min(m0 + n0 + kCols, m_all) - 1) + 1;
          for (int32_t j = fast_div(plan.group_div, min(m0 + n0, m_all - 1)); j < end; ++j)
            if (sees_draft(a.seqs.mask + (int64_t)(g.row0 + j) * a.seqs.mask_words, j, k)) s |= columns(j, j + 1);
          return s;
        }
        s = columns(0, g.rows);
        if (a.window > 0 && t >= a.n_first) {
#pragma unroll 1
          for (int i = 0; i < kCols; ++i)
            if (C.depth[n0 + i] - k >= a.window) s &= ~(1u << i);
        }
        return s;
      };
      uint64_t sum2[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) sum2[i] = 0ull;
      jg0 = jg;
      if (g.n > 0) {  // what the other warps have left of the part's rows
        warp_wait(sm32(&C.q_full), loaded & 1u, lim, abort_flag);
        __syncwarp();
        ++loaded;
      }
      for (int j = 0; j < g.n; ++j, ++jg) {
        if (G::kTurns && (int)(jg & 1u) != w) continue;
        const uint32_t b = jg % (uint32_t)G::kS, sc = lane_base + G::kSCol + b * G::kN + n0;
        const int32_t tile = g.tile(j);
        const bool masked = is_masked(tile);
        const uint32_t see = masked ? sees(tile * kC8T + tk) : 0xFFFFFFFFu;
        warp_wait(sm32(&C.s_full[b]), (jg / (uint32_t)G::kS) & 1u, lim, abort_flag);
        tc_fence_after();
        __syncwarp();
        float ks = C.scales[jg % G::kAhead][0][tk >> 4], vs = C.scales[jg % G::kAhead][1][tk >> 4];
        if (!(ks >= 0.f && ks < INFINITY && vs >= 0.f && vs < INFINITY)) {
          if (see != 0u) report_error(a.status, kErrNonFinite, g.s);
          ks = vs = 0.f;
        }
        const float vx = fmaxf(vs, kC8Least);
        const bool p_free = jg < 2 || mbar_test(sm32(&C.pv_done[(jg - 2u) % G::kPv]), ((jg - 2u) / G::kPv) & 1u);
        uint8_t *const p_tile = c8_shared + G::kPOff + (jg & 1u) * G::kBox;
        float x[kCols];
        // Twice where references move: of the rows whose largest w of this tile is over 2^15,
        // or of all in a part's first tile.
        for (bool move = j < G::kOs;; move = true) {
          // Logits in log2 units, rounded as they are: a reference taken from them is then met
          // exactly, however large they are.
          const uint64_t ks2 = pair_f32(ks, ks), sixteenth = pair_f32(0.0625f, 0.0625f);
          uint32_t hi[kCols], lo[kCols];
          tmem_cols<kCols>(sc, hi);
          tmem_cols<kCols>(sc + R, lo);
          tmem_ready<kCols>(hi);
          tmem_ready<kCols>(lo);
#pragma unroll
          for (int i = 0; i < kCols; i += 2) {
            const uint64_t s2 = fma2(pair_f32(__uint_as_float(lo[i]), __uint_as_float(lo[i + 1])), sixteenth,
                                     pair_f32(__uint_as_float(hi[i]), __uint_as_float(hi[i + 1])));
            const uint64_t f2 = pair_f32(C.factor[n0 + i], C.factor[n0 + i + 1]);
            unpair_f32(mul2(mul2(s2, ks2), f2), x[i], x[i + 1]);
          }
          if (move) {
            const float lv = lg2(vx);
            float l[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) l[i] = ((see >> i) & 1u) ? x[i] + lv : -INFINITY;
            const float top = over_lanes<kCols>(l, lane, [](float p, float q) { return fmaxf(p, q); });
            // the warps' maxima meet in this group's bytes of the tile's P, which is written later
            if (!__all_sync(0xffffffffu, p_free)) wait_pv(jg - 2);
            __syncwarp();
            auto spot = [&](int q, int i) {
              const int row = q * 32 + i;
              return reinterpret_cast<float *>(p_tile + row * 128 + (((n0 >> 4) ^ (row & 7)) << 4));
            };
            if (lane % (32 / kCols) == 0) *spot(wq, lane / (32 / kCols)) = top;
            group_sync(w);
            if (tk < kCols) {
              // the largest, and the least of the warps' largest (of those that see a token)
              float most = -INFINITY, least = INFINITY;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float one = *spot(q, tk);
                most = fmaxf(most, one);
                least = fminf(least, one == -INFINITY ? INFINITY : one);
              }
              const float was = -less_ref[tk], now = most - kC8Head - fminf(fmaxf(most - least - kC8Gap, 0.f), kC8Lift);
              const bool moves = most > was + 15.f;
              alpha[tk] = moves ? ex2(was - now) : 1.f;
              if (moves) less_ref[tk] = -now;
            }
            group_sync(w);
            if (j >= G::kOs) {  // O and the sums hold the earlier tiles of this part
#pragma unroll
              for (int i = 0; i < kCols / 2; ++i) sum2[i] = mul2(sum2[i], pair_f32(alpha[2 * i], alpha[2 * i + 1]));
              wait_pv(jg - G::kOs);
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < kCols; ++i) {
                const float by = alpha[i];
                if (by != 1.f) tmem_scale<G::kHalves, G::kThree ? 3 : 2>(my_o + i, G::kON, R, by);
              }
              tmem_wait_st();
            }
          }
          // exp of the logits relative to the references
#pragma unroll
          for (int i = 0; i < kCols; i += 2) {
            float lo, hi;
            unpair_f32(add2(pair_f32(x[i], x[i + 1]), pair_f32(less_ref[i], less_ref[i + 1])), lo, hi);
            x[i] = ex2(lo);
            x[i + 1] = ex2(hi);
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if (!((see >> i) & 1u)) x[i] = 0.f;
          }
          float most = 0.f;
#pragma unroll
          for (int i = 0; i < kCols; i += 2) most = max3(most, x[i], x[i + 1]);
          if (move || !any_of_group(w, most * vx > kC8Most)) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm32(&C.s_free[b]));
        if (!__all_sync(0xffffffffu, p_free)) wait_pv(jg - 2);  // P's buffer is free
        // The rows of P that are this token's: the group's bytes of its terms.  The sums keep
        // 32 bits, as lse has to; the weights go to the three terms above.
        uint8_t *const prow = p_tile + tk * 128, *const third = R < 64 ? prow : c8_shared + G::kLoBox + tk * 128;
        auto place = [&](uint8_t *row, int col) { return row + (((col >> 4) ^ (tk & 7)) << 4); };
        constexpr int kPut = kCols < 16 ? kCols : 16;  // columns at once
        const uint64_t vs2 = pair_f32(vs, vs);
#pragma unroll
        for (int c = 0; c < kCols; c += kPut) {
          uint32_t ph[kPut / 4], pm[kPut / 4], pl[kPut / 4];
#pragma unroll
          for (int i = 0; i < kPut; i += 4) {
            uint32_t h[2], m[2], l[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint64_t p2 = pair_f32(x[c + i + 2 * k], x[c + i + 2 * k + 1]);
              float w0, w1;
              unpair_f32(mul2(p2, vs2), w0, w1);
              split_e5m2(w0, w1, h[k], m[k], l[k]);
              sum2[(c + i) / 2 + k] = add2(sum2[(c + i) / 2 + k], p2);
            }
            ph[i / 4] = __byte_perm(h[0], h[1], 0x7531);
            pm[i / 4] = __byte_perm(m[0], m[1], 0x7531);
            pl[i / 4] = __byte_perm(l[0], l[1], 0x7531);
          }
          if constexpr (kPut == 8) {
            *reinterpret_cast<uint4 *>(place(prow, 0)) = make_uint4(ph[0], ph[1], pm[0], pm[1]);
            *reinterpret_cast<uint4 *>(place(prow, 16)) = make_uint4(pl[0], pl[1], 0u, 0u);
          } else {
            *reinterpret_cast<uint4 *>(place(prow, n0 + c)) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
            *reinterpret_cast<uint4 *>(place(prow, R + n0 + c)) = make_uint4(pm[0], pm[1], pm[2], pm[3]);
            *reinterpret_cast<uint4 *>(place(third, (R < 64 ? 2 * R : (int)(jg & 1u) * 64) + n0 + c)) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
          }
        }
        if (masked && veiled) {
          // A NaN of V would reach, as 0 x NaN, the rows that do not see its token: it is
          // cleared here and given to the rows that do see it when the output is written.
          // (The slot's earlier copy is known to have landed once P V of the tile before the
          // last is done.)
          const uint32_t at = ns + (uint32_t)c8_v_pos(j, g.n), slot = at % G::kSlots;
          warp_wait(sm32(&C.full[slot]), (at / G::kSlots) & 1u, lim, abort_flag);
          __syncwarp();
          uint4 *vt = reinterpret_cast<uint4 *>(c8_shared + G::kRingOff + slot * G::kSlot);
          for (int i = G::kTurns ? tk : tid; i < (int)(G::kSlot / 16); i += 32 * G::kSoft / G::kOs) {
            const uint4 y = vt[i];
            uint32_t e[4] = {y.x, y.y, y.z, y.w}, hit = 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) hit |= ((e[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // a byte's seven bits all set
            if (hit != 0u) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t z = ((e[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                e[k] &= ~((z >> 7) * 0xFFu);
              }
              vt[i] = make_uint4(e[0], e[1], e[2], e[3]);
              *reinterpret_cast<volatile int32_t *>(&C.bad[seg & 1]) = seg;
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm32(&C.p_ready[jg & 1u]));
      }
      ns += (uint32_t)(2 * g.n);
      more = advance(next);
      if (more && next.n > 0) fetch_q(next);
      bool fix = false;
      if (g.n > 0) {  // S and P V of every tile are done: Q may go, O may be read
        if (G::kTurns && g.n > 1) wait_pv(jg - 2);
        wait_pv(jg - 1);
        tc_fence_after();
        __syncwarp();
        fix = *reinterpret_cast<volatile int32_t *>(&C.bad[seg & 1]) == seg;
      }
      if (fix) {  // rare: the rows of this thread's dims that see a cleared NaN
        const int first = w * (R / G::kGroups);
#pragma unroll 1
        for (int n = first; n < first + R / G::kGroups && m0 + n < m_all; ++n) {
          const int32_t j = fast_div(plan.group_div, m0 + n);
          const uint32_t *mrow = chain ? nullptr : a.seqs.mask + (int64_t)(g.row0 + j) * a.seqs.mask_words;
          const int32_t at = g.ctx + (chain ? j : C.depth[n]);
#pragma unroll 1
          for (int h = 0; h < G::kHalves; ++h) {
            bool hit = false;
            for (int i = 0; i < g.n; ++i) {
              const int32_t t0 = g.tile(i) * kC8T;
              if (!is_masked(g.tile(i))) continue;
              for (int32_t t = t0; t < min(kv, t0 + kC8T); ++t) {
                const bool drafted = t >= g.ctx;
                if (drafted && !sees_draft(mrow, j, t - g.ctx)) continue;
                if (a.window > 0 && t >= a.n_first && at - t >= a.window && (chain || !drafted)) continue;
                const int64_t slot = token_slot(a.seqs, g.s, t);
                hit = hit || (slot >= 0 && nan8(a.v_pool[(slot * a.nkv + g.kvh) * HD + h * 128 + tk]));
              }
            }
            __syncwarp();
            tmem_scale1(lane_base + (has(0) ? 0u : G::kOCols) + (uint32_t)(h * G::kON + n), hit ? NAN : 1.f);
          }
        }
        tmem_wait_st();
      }
      const int64_t part = (int64_t)blockIdx.x * 2 + ((g.flags & C8Seg::kHead) ? 0 : 1);
      const bool whole = (g.flags & C8Seg::kWhole) != 0;
      float(*const sums)[kCols] = reinterpret_cast<float(*)[kCols]>(c8_shared + G::kPOff);  // P is read
      if (!empty) {
        // the rows' sums over this group's threads, in a fixed order
        float sum[kCols];
#pragma unroll
        for (int i = 0; i < kCols; i += 2) unpair_f32(sum2[i / 2], sum[i], sum[i + 1]);
        const float mine = over_lanes<kCols>(sum, lane, [](float p, float q) { return p + q; });
        if (lane % (32 / kCols) == 0) sums[warp][lane / (32 / kCols)] = mine;
      }
      soft_sync(32 * G::kSoft);
      if (!empty && tid < R) {
        const int n = tid;
        float ref = kC8Unset, all = 0.f;
        auto sum_of = [&](int o, int i) { return (sums[4 * o][i] + sums[4 * o + 1][i]) + (sums[4 * o + 2][i] + sums[4 * o + 3][i]); };
        if constexpr (G::kTurns) {
          const float r0 = has(0) ? -C.less_ref[n] : kC8Unset, r1 = has(1) ? -C.less_ref[kCols + n] : kC8Unset;
          ref = fmaxf(r0, r1);
          const float by0 = ex2(r0 - ref), by1 = ex2(r1 - ref);
          C.mix[n] = by0;
          C.mix[kCols + n] = by1;
          if (has(0)) all = sum_of(0, n) * by0;
          if (has(1)) all = fmaf(sum_of(1, n), by1, all);
        } else if (g.n > 0) {
          ref = -C.less_ref[n];
          all = sum_of(n / kCols, n % kCols);
        }
        inverse[n] = !whole ? 1.f : all == 0.f ? 0.f : rcp(all);
        int64_t where = -1;
        if (m0 + n < m_all) {
          const int32_t j = fast_div(plan.group_div, m0 + n), head = g.kvh * a.group + (m0 + n - j * a.group);
          where = whole ? (int64_t)(g.row0 + j) * a.out_stride + (int64_t)head * HD : (part * R + n) * HD;
          if (!whole) part_ml[part * R + n] = make_float2(ref, all);
          else if (a.lse)
            a.lse[(int64_t)(g.row0 + j) * a.nq + head] = all == 0.f ? -INFINITY : lse_of(ref, all);
        }
        C.where[n] = where;
      }
      soft_sync(32 * G::kSoft);  // the part's references and sums are read
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && found.share.n > 0 && (C.abort || !laid_out)) report_error(a.status, kErrTimeout, found.seq);
  if (warp == G::kMmaS)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// Joins the parts of the units that several CTAs share.  A block has the unit that one CTA
// ended with, if it did; a warp a row of it, 4 dims a lane and half, and every kGroups-th part; the
// groups' results are then added in order.  (A warp for every row of the call, which looked
// its unit up, took 23 us of a chunk of 2048 rows' 210.)  Units and parts are written while this
// launch is already resident, so they are no __restrict__ arguments: nothing may read them ahead
// of the wait.
// Four warps of 64 registers are what the SM has left beside a CTA of 8 rows, so that they wait
// there while it runs (of eight, which start when it ends: decode of 16 rows 106.6 us, 104.6
// with four; in a window of 4096 24.6 and 23.4; one row of 65535 tokens 25.7 and 24.4).
constexpr int kC8JoinWarps = 4;

template <int HD, int R, int kGroups>
__global__ void __launch_bounds__(32 * kC8JoinWarps)
cache8_join_kernel(const Cache8Args a, const C8Plan plan, int32_t ctas, const C8Open *open, const float2 *part_ml, const float4 *part_o) {
  constexpr int kQuads = HD / 128;
  __shared__ float4 acc_s[kGroups > 1 ? kC8JoinWarps : 1][kQuads][32];
  __shared__ float2 ml_s[kGroups > 1 ? kC8JoinWarps : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = warp % kGroups;
  grid_dependency_sync();
  // The units are those that CTAs ended with, a block's own CTA's or, where there are fewer
  // blocks, the nth that there is.  (As many as there can be, but for sequences that overlap.)
  for (int32_t nth = blockIdx.x;; nth += (int32_t)gridDim.x) {
    int32_t from = nth < ctas ? nth : -1;
    if (gridDim.x < (uint32_t)ctas) {
      int32_t last[kC8MaxCtas / 32], left = nth;
#pragma unroll
      for (int i = 0; i < kC8MaxCtas / 32; ++i) last[i] = 32 * i + lane < ctas ? open[32 * i + lane].last : -1;
      from = -1;
#pragma unroll
      for (int i = 0; i < kC8MaxCtas / 32; ++i) {
        const uint32_t has = __ballot_sync(0xffffffffu, last[i] >= 0);
        const uint32_t it = __ballot_sync(0xffffffffu, last[i] >= 0 && __popc(has & ((1u << lane) - 1u)) == left);
        if (it != 0u) from = 32 * i + __ffs(it) - 1;
        left -= __popc(has);
      }
    }
    if (from < 0) return;
    const int32_t rank = from & ((1 << plan.head_log) - 1), c0 = from >> plan.head_log;
    const C8Open unit = open[from];
    const int32_t c1 = unit.last;  // the team of the last part
    if (c1 < 0) continue;
    const int32_t r = (int32_t)blockIdx.y * (kC8JoinWarps / kGroups) + warp / kGroups;
    const bool mine = unit.m0 + r < unit.rows * a.group;
    const int32_t j = mine ? fast_div(plan.group_div, unit.m0 + r) : 0, row = unit.row0 + j;
    const int32_t head = unit.kvh * a.group + (unit.m0 + r - j * a.group);
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
          const int64_t part = (((int64_t)min(at, c1) << plan.head_log) + rank) * 2 + (min(at, c1) == c0 ? 1 : 0);
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
      const int first = warp - grp;
      top = -INFINITY;
      for (int g = 0; g < kGroups; ++g) top = fmaxf(top, ml_s[first + g].x);
      const float use = top == -INFINITY ? 0.f : top;
      all = 0.f;
#pragma unroll
      for (int i = 0; i < kQuads; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int g = 0; g < kGroups && grp == 0; ++g) {
        if (ml_s[first + g].x == -INFINITY) continue;
        const float by = ex2(ml_s[first + g].x - use);
        all = fmaf(ml_s[first + g].y, by, all);
#pragma unroll
        for (int i = 0; i < kQuads; ++i) add(acc[i], acc_s[first + g][i][lane], by);
      }
    }
    if constexpr (kGroups > 1) __syncthreads();  // read before the next unit's
    if (!mine || grp != 0) continue;
    const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll
    for (int i = 0; i < kQuads; ++i)
      *reinterpret_cast<uint2 *>(a.out + (int64_t)row * a.out_stride + (int64_t)head * HD + 128 * i + 4 * lane) =
          make_uint2(pack_f32_bf16(acc[i].x * inv, acc[i].y * inv), pack_f32_bf16(acc[i].z * inv, acc[i].w * inv));
    if (lane == 0 && a.lse)
      a.lse[(int64_t)row * a.nq + head] = all == 0.f ? -INFINITY : lse_of(top, all);
  }
}

// The workspace: the units that CTAs end with, the parts' (ref, sum) and O.
int64_t rows_of_part(int64_t n_rows, int32_t group) {
  int64_t r = 8;
  while (r < kC8MostRows && r < n_rows * group) r *= 2;
  return r;
}
constexpr int64_t kC8OpenBytes = (kC8MaxCtas * (int64_t)sizeof(C8Open) + 255) / 256 * 256;
int64_t ml_bytes(int64_t rows) { return (int64_t)kC8MaxCtas * 2 * rows * 8; }
int64_t o_bytes(int64_t rows, int32_t head_dim) { return (int64_t)kC8MaxCtas * 2 * rows * head_dim * 4; }

template <int HD, int R>
cudaError_t launch_rows(const Cache8Args &a, cudaStream_t stream) {
  static PerDevice smem_attr;
  const cudaError_t e = set_smem_once(smem_attr, cache8_attn_kernel<HD, R>, c8_smem<HD, R>());
  if (e != cudaSuccess) return e;
  uint8_t *ws = static_cast<uint8_t *>(a.ws);
  C8Open *open = reinterpret_cast<C8Open *>(ws);
  float2 *ml = reinterpret_cast<float2 *>(ws + kC8OpenBytes);
  float *o = reinterpret_cast<float *>(ws + kC8OpenBytes + ml_bytes(R));
  // KV heads side by side read neighbouring pieces of the same rows.
  int head_log = 0;
  while (head_log < 3 && a.nkv % (2 << head_log) == 0) ++head_log;
  const int ctas = ((device_sm_count() < kC8MaxCtas ? device_sm_count() : kC8MaxCtas) >> head_log) << head_log;
  const C8Plan plan = {make_fast_div(a.group), head_log, R / a.group + 2};
  cudaError_t r = launch_dependent(cache8_attn_kernel<HD, R>, dim3((unsigned)ctas), dim3(C8Geom<HD, R>::kThreads), c8_smem<HD, R>(), stream, 1u, a,
                                   plan, open, ml, o);
  // a table of one tile leaves no unit to share
  if (r != cudaSuccess || (int64_t)a.seqs.table_len * a.seqs.page.d <= kC8T) return r;
  // One group of parts per warp where units outnumber the CTAs (few parts each), a CTA's
  // where a unit spreads over many.  A block for every CTA, or for as many units as there can
  // be, where the rows of more would be thousands of blocks (64 rows over 65k tokens 118 us, 112;
  // but one row over 515 9.7 us, 10.5 where it has to find its unit).
  const int64_t rows = (int64_t)a.seqs.n_rows * a.group, units = (int64_t)a.nkv * ((rows + R - 1) / R);
  const int64_t open_most = (int64_t)a.nkv * (a.seqs.n_seqs + rows / R);
  const bool many = ctas >= 8 * units;
  return launch_dependent(many ? cache8_join_kernel<HD, R, kC8JoinWarps> : cache8_join_kernel<HD, R, 1>,
                          dim3((unsigned)(R > 8 && open_most < ctas ? open_most : ctas), many ? R : R / kC8JoinWarps), dim3(32 * kC8JoinWarps), 0,
                          stream, 1u, a, plan, ctas, open, ml, reinterpret_cast<const float4 *>(o));
}

// The rows of a unit.  Enough for a sequence's rows by the call's mean, as a tile of 64 costs
// 1.46 us of a CTA where one of 32 costs 0.89, of 16 0.79 and of 8 0.73 (heads of 256, from L2).
// Fewer where the GPU would stand idle meanwhile: a unit of 64 takes some 10 us besides its
// tiles, one of 8 2 us.  So by how many tiles of units of 64 a CTA would get at most, with 3
// tiles for a unit's beginning: the bounds are fitted with that, c8_start() is what balances CTAs
// that have many.  8, 16, 32, 64 rows a unit, and the rule's choice under a table of 65536 tokens
// a sequence (us, in a graph): without a window the bound is the table's, which the host knows,
// not the contexts', so that a long one gets the mean's units.
//   0.4  2 sequences of 10 rows, 16 heads over 2, a window of 199     13.0  14.5  16.2  18.1  13
//   0.9  4 of 24, 16 over 2, 300 tokens                               18.9  16.5  17.5  19.9  20
//   1.0  1 of 64, 16 over 2, 600 tokens                               18.2  16.7  17.7  20.2  20
//   1.4  1 of 24, 16 over 2, 4000 tokens                              20.6  20.8  18.6  20.6  21
//   2.5  4 of 64, 16 over 2, 300 tokens                               29.8  24.4  16.5  19.5  20
//   3.3  6 of 112, 16 over 2, 22 to 139 tokens                        51.0  38.1  32.8  31.4  31
//   8.9  17 of 95, 12 over 4, 8 tokens                                84.6  57.5  44.2  36.5  40
int32_t rows_of_unit(const Cache8Args &a, int64_t most) {
  const int64_t n = a.seqs.n_seqs, mean = ((int64_t)a.seqs.n_rows * a.group + n - 1) / n;
  const int64_t all = (most + kC8T - 1) / kC8T;
  const int64_t near = a.window > 0 ? ((int64_t)a.n_first + kC8T - 1) / kC8T + ((int64_t)a.window + kC8T - 1) / kC8T + 1 : all;
  const int64_t work = n * a.nkv * ((mean + 63) / 64) * ((all < near ? all : near) + 3), ctas = device_sm_count();
  const int32_t by_work = 2 * work <= ctas ? 8 : 5 * work <= 6 * ctas ? 16 : work <= 3 * ctas ? 32 : 64;
  const int32_t by_mean = mean <= 8 ? 8 : mean <= 16 ? 16 : mean <= 32 ? 32 : 64;
  return by_work < by_mean ? by_work : by_mean;
}

template <int HD>
cudaError_t launch_hd(const Cache8Args &args, cudaStream_t stream) {
  Cache8Args a = args;
  const int64_t most = (int64_t)a.seqs.table_len * a.seqs.page.d;  // (below 2^31 - 256)
  if (a.window >= most) a.window = 0;  // no cached token is that far back
  a.n_first = a.window == 0 ? 0 : (int32_t)(a.n_first < most ? a.n_first : most);
  const int32_t rows = rows_of_unit(a, most);
  return rows == 8    ? launch_rows<HD, 8>(a, stream)
         : rows == 16 ? launch_rows<HD, 16>(a, stream)
         : rows == 32 ? launch_rows<HD, 32>(a, stream)
                      : launch_rows<HD, 64>(a, stream);
}

}  // namespace

int64_t cache8_workspace_bytes(int32_t n_rows, int32_t group, int32_t head_dim) {
  const int64_t rows = rows_of_part(n_rows, group);
  return kC8OpenBytes + ml_bytes(rows) + o_bytes(rows, head_dim);
}

cudaError_t launch_cache8_attn(const Cache8Args &a, int32_t head_dim, cudaStream_t stream) {
  return head_dim == 256 ? launch_hd<256>(a, stream) : launch_hd<128>(a, stream);
}

}  // namespace qsa
