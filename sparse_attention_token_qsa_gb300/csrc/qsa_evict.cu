// The tokens a shortened cache keeps: the units (1 or 4 tokens) of the largest
// accumulated attention mass, the first and the last ones always among them.
//
// A unit's mass is the f32 sum of its tokens' in token order, a token's the
// f32 sum over the KV heads in head order; units are ordered by mass
// descending, then index ascending (-0 equals +0).
//
// One thread-block cluster per sequence, a contiguous run of units per CTA.  The
// mass is read once, into monotonic 32-bit keys in shared memory; three radix
// rounds (11, 11 and 10 bits) find the key of the last unit that stays.  Over a
// cluster the bins are searched in two steps, sums of 32 and then 32 bins, read
// over distributed shared memory: reading all 2048 of every CTA took 2100 cycles a
// round, the two reads 1600.  Exact zeros, which a cache is full of, are summed
// over the warp and not by atomics on one bin.  A unit's place in the list follows
// from two counts before it, larger keys and equal ones (of which the first `ties`
// stay), taken per warp over its own run: no barrier while the list is written.
//
// 32 caches of 131k-262k tokens (48 MB of mass) take 21 us, 34 % of the copy
// bandwidth: 5.5 us of them read the mass, the rest is the chain of rounds, their
// barriers and the list.  A cache of 4099 tokens takes 5 us, all of it that chain.
#include <cooperative_groups.h>

#include "qsa_launch.h"
#include "qsa_paged.cuh"
#include "qsa_select_util.cuh"

namespace qsa {

namespace {

namespace cg = cooperative_groups;

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;          // of the first two rounds; the last has 1024
constexpr int kEvMaxKeys = 49152;      // per CTA, in shared memory
constexpr int kEvMaxCluster = 8;
constexpr int kEvBatch = 4;            // loads of 16 bytes a thread has on their way for each KV head
constexpr int kEvGroup = 32;           // bins that a coarse one sums

struct EvictCtrl {
  uint32_t hist[3][kEvBins];
  uint32_t coarse[3][kEvBins / kEvGroup];
  uint32_t warp_tot[kEvWarps], gt[kEvWarps], eq[kEvWarps];
  uint32_t gt_all, eq_all, above, inside;
  int32_t bin, bad;
};
constexpr size_t kEvKeysOff = (sizeof(EvictCtrl) + 15) / 16 * 16;

__device__ __forceinline__ float4 add4(float4 s, float4 x) {
  return make_float4(__fadd_rn(s.x, x.x), __fadd_rn(s.y, x.y), __fadd_rn(s.z, x.z), __fadd_rn(s.w, x.w));
}

// Keys of four tokens' masses: four units of one token, or one unit of four.
// Returns whether all are finite.
template <int UNIT>
__device__ __forceinline__ bool unit_keys(float4 s, uint32_t (&key)[4 / UNIT], int units) {
  if constexpr (UNIT == 4) {
    const float f = __fadd_rn(__fadd_rn(__fadd_rn(s.x, s.y), s.z), s.w);
    key[0] = order_key(f);
    return isfinite(f);
  } else {
    key[0] = order_key(s.x);
    key[1] = order_key(s.y);
    key[2] = order_key(s.z);
    key[3] = order_key(s.w);
    return isfinite(s.x) && (units <= 1 || isfinite(s.y)) && (units <= 2 || isfinite(s.z)) && (units <= 3 || isfinite(s.w));
  }
}

// The sum of the lanes' x up to this one.
__device__ __forceinline__ uint32_t warp_upto(uint32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// A protected unit's key lies above, the key past the last unit below, that of any
// finite mass: neither needs a test after the first pass.
constexpr uint32_t kProtected = 0xffffffffu, kNoUnit = 0u;

template <int UNIT, bool CACHED>
__global__ void __launch_bounds__(kEvThreads)
evict_kernel(const EvictArgs a, int32_t ctas) {
  extern __shared__ __align__(16) uint8_t ev_smem[];
  EvictCtrl &C = *reinterpret_cast<EvictCtrl *>(ev_smem);
  uint32_t *keys = reinterpret_cast<uint32_t *>(ev_smem + kEvKeysOff);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t s = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  auto all_sync = [&]() {
    if (ctas > 1) cluster.sync();
    else __syncthreads();
  };
  for (int i = tid; i < 3 * kEvBins; i += kEvThreads) (&C.hist[0][0])[i] = 0u;
  if (tid == 0) C.bad = 0;
  grid_dependency_sync();
  const int32_t len = a.length[s];
  if (len < 0 || len > a.tokens) {  // (every CTA of the cluster)
    if (tid == 0 && rank == 0) report_error(a.status, kErrRowRange, s);
    return;
  }
  const int32_t units = len / UNIT, keep = a.keep / UNIT;
  int32_t *sel = a.sel + (int64_t)s * a.sel_cols;
  if (units <= keep) {
    for (int32_t t = rank * kEvThreads + tid; t < len; t += ctas * kEvThreads) sel[t] = t;
    if (tid == 0 && rank == 0) a.n_sel[s] = len;
    return;
  }
  // this CTA's units [u0, u1), a whole number of warp steps of 128
  const int32_t seg = ((units + ctas - 1) / ctas + 127) & ~127;
  const int32_t u0 = min((int64_t)units, (int64_t)rank * seg), u1 = min((int64_t)units, (int64_t)u0 + seg);
  const int32_t lo = a.n_first / UNIT, hi = units - a.n_last / UNIT;  // units in [lo, hi) compete
  const float *m = a.mass + (int64_t)s * a.nkv * a.mass_cols;
  constexpr int kPer = 4 / UNIT;  // units per load
  __syncthreads();

  // ---- round 0 while the mass is read: keys, their upper 11 bits, and what is not finite
  const int32_t loads = ((u1 - u0 + 127) & ~127) / kPer;
  uint32_t zeros = 0;
  bool finite = true;
  for (int32_t i0 = tid; i0 < loads; i0 += kEvBatch * kEvThreads) {
    float4 sum[kEvBatch];
#pragma unroll
    for (int b = 0; b < kEvBatch; ++b) {
      const int32_t u = u0 + (i0 + b * kEvThreads) * kPer;
      sum[b] = u < u1 ? *reinterpret_cast<const float4 *>(m + (int64_t)u * UNIT) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int32_t h = 1; h < a.nkv; ++h) {
      float4 x[kEvBatch];
#pragma unroll
      for (int b = 0; b < kEvBatch; ++b) {
        const int32_t u = u0 + (i0 + b * kEvThreads) * kPer;
        x[b] = u < u1 ? *reinterpret_cast<const float4 *>(m + h * a.mass_cols + (int64_t)u * UNIT) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int b = 0; b < kEvBatch; ++b) sum[b] = add4(sum[b], x[b]);
    }
#pragma unroll
    for (int b = 0; b < kEvBatch; ++b) {
      const int32_t i = i0 + b * kEvThreads, u = u0 + i * kPer;
      if (i >= loads) break;
      uint32_t key[kPer];
      finite = unit_keys<UNIT>(sum[b], key, u1 - u) && finite;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (u + e >= u1) key[e] = kNoUnit;
        else if (u + e < lo || u + e >= hi) key[e] = kProtected;
        else if (key[e] == kZeroKey) ++zeros;
        else atomicAdd(&C.hist[0][key[e] >> 21], 1u);
      }
      if constexpr (CACHED) {
        if constexpr (UNIT == 4) keys[i] = key[0];
        else reinterpret_cast<uint4 *>(keys)[i] = make_uint4(key[0], key[1], key[2], key[3]);
      }
    }
  }
  auto add_zeros = [&](int round, int shift) {
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if (lane == 0 && zeros) atomicAdd(&C.hist[round][(kZeroKey >> shift) & (uint32_t)(kEvBins - 1)], zeros);
    zeros = 0;
  };
  add_zeros(0, 21);
  if (!finite) C.bad = 1;

  // four keys from unit u on (u - u0 a multiple of 4, u < u1)
  auto keys_at = [&](int32_t u) -> uint4 {
    if constexpr (CACHED) {
      return *reinterpret_cast<const uint4 *>(keys + (u - u0));
    } else {
      uint32_t k[4];
#pragma unroll
      for (int e = 0; e < 4; e += kPer) {
        uint32_t key[kPer] = {};
        if (u + e < u1) {
          const float *at = m + (int64_t)(u + e) * UNIT;
          float4 sum = *reinterpret_cast<const float4 *>(at);
          for (int32_t h = 1; h < a.nkv; ++h) sum = add4(sum, *reinterpret_cast<const float4 *>(at + h * a.mass_cols));
          unit_keys<UNIT>(sum, key, kPer);
        }
#pragma unroll
        for (int f = 0; f < kPer; ++f)
          k[e + f] = u + e + f >= u1 ? kNoUnit : u + e + f < lo || u + e + f >= hi ? kProtected : key[f];
      }
      return make_uint4(k[0], k[1], k[2], k[3]);
    }
  };

  // one counter of all the CTAs, every read on its way at once
  auto sum_ctas = [&](uint32_t *counter) -> uint32_t {
    uint32_t part[kEvMaxCluster], sum = 0;
#pragma unroll
    for (int r = 0; r < kEvMaxCluster; ++r) part[r] = r < ctas ? *cluster.map_shared_rank(counter, r) : 0u;
#pragma unroll
    for (int r = 0; r < kEvMaxCluster; ++r) sum += part[r];
    return sum;
  };

  // ---- the key of the last unit that stays: the need-th largest of those that compete
  uint32_t need = (uint32_t)(keep - lo - (units - hi)), prefix = 0;
  const bool none = need == 0;  // the protected units fill the budget
  uint32_t cut = kProtected - 1u;
#pragma unroll
  for (int round = 0; round < 3; ++round) {
    constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
    if (round > 0) {
      for (int32_t u = u0 + 4 * tid; u < u1; u += 4 * kEvThreads) {
        const uint4 k4 = keys_at(u);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((k[e] >> (round == 1 ? 21 : 10)) != prefix) continue;
          if (k[e] == kZeroKey) ++zeros;
          else atomicAdd(&C.hist[round][(k[e] >> kShift[round]) & ((1u << kBits[round]) - 1u)], 1u);
        }
      }
      add_zeros(round, kShift[round]);
    }
    if (ctas > 1) {
      __syncthreads();
#pragma unroll
      for (int g = 2 * warp; g < 2 * warp + 2; ++g) {
        const uint32_t n = __reduce_add_sync(0xffffffffu, C.hist[round][g * kEvGroup + lane]);
        if (lane == 0) C.coarse[round][g] = n;
      }
    }
    all_sync();  // every CTA's histogram (and, in round 0, its verdict) is there
    if (round == 0) {
      bool bad = C.bad != 0;
      if (ctas > 1) bad = __any_sync(0xffffffffu, lane < ctas && *cluster.map_shared_rank(&C.bad, lane < ctas ? lane : 0) != 0);
      if (bad) {  // the same in every CTA, none of which may leave while it is read
        if (tid == 0 && rank == 0) report_error(a.status, kErrNonFinite, s);
        all_sync();
        return;
      }
      if (none) break;
    }
    if (ctas == 1) {  // the bins from the top, two a thread
      const int at = kEvBins / 2 - 1 - tid;
      const uint2 n = reinterpret_cast<const uint2 *>(C.hist[round])[at];
      uint32_t upto = warp_upto(n.x + n.y, lane);
      if (lane == 31) C.warp_tot[warp] = upto;
      __syncthreads();
      upto += __reduce_add_sync(0xffffffffu, lane < warp ? C.warp_tot[lane] : 0u);
      const uint32_t above = upto - n.x - n.y;
      if (above < need && need <= upto) {  // one thread's
        const bool upper = need <= above + n.y;
        C.bin = 2 * at + (upper ? 1 : 0);
        C.above = upper ? above : above + n.y;
        C.inside = upper ? n.y : n.x;
      }
    } else if (warp == 0) {
      // One warp looks through the 64 groups and then the 32 bins of one: reading all
      // the bins of the other CTAs takes longer than its chain of two reads.
      uint32_t upper = sum_ctas(&C.coarse[round][63 - lane]), lower = sum_ctas(&C.coarse[round][31 - lane]);
      uint32_t up = warp_upto(upper, lane);
      const uint32_t low = warp_upto(lower, lane) + __shfl_sync(0xffffffffu, up, 31);
      uint32_t hit = __ballot_sync(0xffffffffu, up >= need);
      const bool in_upper = hit != 0;
      if (!in_upper) {
        up = low;
        upper = lower;
        hit = __ballot_sync(0xffffffffu, low >= need);
      }
      int src = (__ffs(hit) - 1) & 31;
      const int at = ((in_upper ? 63 : 31) - src) * kEvGroup + 31 - lane;
      const uint32_t n = sum_ctas(&C.hist[round][at]);
      up = __shfl_sync(0xffffffffu, up - upper, src) + warp_upto(n, lane);
      hit = __ballot_sync(0xffffffffu, up >= need);
      src = (__ffs(hit) - 1) & 31;
      if (lane == src) {
        C.bin = at;
        C.above = up - n;
        C.inside = n;
      }
    }
    __syncthreads();
    prefix = (prefix << kBits[round]) | (uint32_t)C.bin;
    need -= C.above;
    // Where the whole bin stays, every key from its lowest on does, and no bit more is
    // needed: after two rounds that is the rule, keys that share 22 bits being few.
    if (round < 2 && need == C.inside) {
      cut = (prefix << (round == 0 ? 21 : 10)) - 1u;
      need = 0;
      break;
    }
    if (round == 2) cut = prefix;
  }
  const uint32_t ties = none ? 0u : need;

  // ---- counts before each warp's run, then the list
  const bool wide = (reinterpret_cast<uintptr_t>(a.sel) & 15u) == 0 && (a.sel_cols & 3) == 0;
  auto put = [&](uint32_t at, int32_t u) {
    int32_t *to = sel + (int64_t)at * UNIT;
    const int32_t tok = u * UNIT;
    if (UNIT == 4 && wide) {
      *reinterpret_cast<int4 *>(to) = make_int4(tok, tok + 1, tok + 2, tok + 3);
    } else {
#pragma unroll
      for (int f = 0; f < UNIT; ++f) to[f] = tok + f;
    }
  };
  // Keys in shared memory: a lane takes `lane_run` units side by side, an odd number,
  // which no two lanes read from one bank; what stays of them are the bits of two words.
  // Otherwise a warp takes steps of 128 units, twice.
  const int32_t lane_run = ((seg + kEvThreads - 1) / kEvThreads) | 1;
  const int32_t run = CACHED ? 32 * lane_run : ((seg + kEvWarps - 1) / kEvWarps + 127) & ~127;
  const int32_t w0 = min((int64_t)u1, (int64_t)u0 + warp * run), w1 = min((int64_t)u1, (int64_t)w0 + run);
  uint32_t gt = 0, eq = 0;
  uint64_t gt_bits = 0, eq_bits = 0;
  if constexpr (CACHED) {
    const int32_t l0 = w0 + lane * lane_run, n = min(lane_run, w1 - l0);
#pragma unroll 4
    for (int32_t i = 0; i < n; ++i) {
      const uint32_t k = keys[l0 - u0 + i];
      gt_bits |= (uint64_t)(k > cut) << i;
      eq_bits |= (uint64_t)(k == cut) << i;
    }
    gt = __popcll(gt_bits);
    eq = __popcll(eq_bits);
  } else {
    for (int32_t u = w0 + 4 * lane; u < w1; u += 128) {
      const uint4 k = keys_at(u);
      gt += (k.x > cut) + (k.y > cut) + (k.z > cut) + (k.w > cut);
      eq += (k.x == cut) + (k.y == cut) + (k.z == cut) + (k.w == cut);
    }
  }
  const uint32_t lane_gt = gt, lane_eq = eq;
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    C.gt[warp] = gt;
    C.eq[warp] = eq;
  }
  __syncthreads();
  const uint32_t w_gt = C.gt[lane], w_eq = C.eq[lane];
  gt = __reduce_add_sync(0xffffffffu, lane < warp ? w_gt : 0u);
  eq = __reduce_add_sync(0xffffffffu, lane < warp ? w_eq : 0u);
  if (ctas > 1) {
    if (warp == 0) {
      const uint32_t gt_all = __reduce_add_sync(0xffffffffu, w_gt), eq_all = __reduce_add_sync(0xffffffffu, w_eq);
      if (lane == 0) {
        C.gt_all = gt_all;
        C.eq_all = eq_all;
      }
    }
    cluster.sync();
    const bool before = lane < rank;
    gt += __reduce_add_sync(0xffffffffu, before ? *cluster.map_shared_rank(&C.gt_all, before ? lane : 0) : 0u);
    eq += __reduce_add_sync(0xffffffffu, before ? *cluster.map_shared_rank(&C.eq_all, before ? lane : 0) : 0u);
    cluster.sync();  // no CTA leaves while its counts are read
  }
  if constexpr (CACHED) {
    uint32_t my_gt = gt + warp_upto(lane_gt, lane) - lane_gt, my_eq = eq + warp_upto(lane_eq, lane) - lane_eq;
    const int32_t l0 = w0 + lane * lane_run;
    for (uint64_t stay = gt_bits | eq_bits; stay; stay &= stay - 1) {
      const int i = __ffsll((long long)stay) - 1;
      const bool more = (gt_bits >> i) & 1u;
      if (more || my_eq < ties) put(my_gt + min(my_eq, ties), l0 + i);
      my_gt += more;
      my_eq += !more;
    }
  } else
  for (int32_t b = w0; b < w1; b += 128) {
    const int32_t u = b + 4 * lane;
    const uint4 k4 = u < w1 ? keys_at(u) : make_uint4(kNoUnit, kNoUnit, kNoUnit, kNoUnit);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    uint32_t mine = 0;  // larger keys in the lower half, equal ones in the upper
#pragma unroll
    for (int e = 0; e < 4; ++e) mine += k[e] > cut ? 1u : k[e] == cut ? 0x10000u : 0u;
    if (!__any_sync(0xffffffffu, mine != 0)) continue;
    const uint32_t upto = warp_upto(mine, lane), all = __shfl_sync(0xffffffffu, upto, 31);
    uint32_t my_gt = gt + ((upto - mine) & 0xffffu), my_eq = eq + ((upto - mine) >> 16);
    gt += all & 0xffffu;
    eq += all >> 16;
    if (mine == 0) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool more = k[e] > cut, same = k[e] == cut;
      if (more || (same && my_eq < ties)) {
        put(my_gt + min(my_eq, ties), u + e);
      }
      my_gt += more;
      my_eq += same;
    }
  }
  if (rank == 0) {  // the tokens past the last whole unit
    if (tid < len - units * UNIT) sel[(int64_t)keep * UNIT + tid] = units * UNIT + tid;
    if (tid == 0) a.n_sel[s] = a.keep + len - units * UNIT;
  }
}

template <int UNIT, bool CACHED>
cudaError_t launch_evict(const EvictArgs &a, int32_t n_seqs, int32_t ctas, int32_t keys, cudaStream_t stream) {
  static PerDevice smem_attr;
  const cudaError_t e = set_smem_once(smem_attr, evict_kernel<UNIT, CACHED>, kEvKeysOff + (size_t)(CACHED ? kEvMaxKeys : 0) * 4);
  if (e != cudaSuccess) return e;
  return launch_dependent(evict_kernel<UNIT, CACHED>, dim3((unsigned)(n_seqs * ctas)), dim3(kEvThreads),
                          kEvKeysOff + (size_t)(CACHED ? keys : 0) * 4, stream, (unsigned)ctas, a, ctas);
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs &a, int32_t n_seqs, cudaStream_t stream) {
  const int32_t units = a.tokens / a.unit;
  // CTAs per sequence: doubled while a run is longer than 4096 units and the launch
  // still has an SM for each, or while a run does not fit shared memory
  int32_t ctas = 1;
  while (ctas < kEvMaxCluster && (units / ctas > kEvMaxKeys - 128 ||
                                  (units / ctas > 4096 && (int64_t)n_seqs * ctas * 2 <= (int64_t)device_sm_count())))
    ctas *= 2;
  const int32_t keys = ((units + ctas - 1) / ctas + 127) & ~127;
  if (a.unit == 4)
    return keys <= kEvMaxKeys ? launch_evict<4, true>(a, n_seqs, ctas, keys, stream)
                              : launch_evict<4, false>(a, n_seqs, ctas, keys, stream);
  return keys <= kEvMaxKeys ? launch_evict<1, true>(a, n_seqs, ctas, keys, stream)
                            : launch_evict<1, false>(a, n_seqs, ctas, keys, stream);
}

}  // namespace qsa
