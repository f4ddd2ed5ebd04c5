// The tokens a shortened cache keeps: the units (1 or 4 tokens) of the largest
// accumulated attention mass, the first and the last ones always among them.
//
// A unit's mass is the f32 sum of its tokens' in token order, a token's the
// f32 sum over the KV heads in head order; units are ordered by mass
// descending, then index ascending (-0 equals +0).
//
// One thread-block cluster per sequence, a contiguous run of units per CTA.  The
// mass is read once, into monotonic 32-bit keys in shared memory; three radix
// rounds (11, 11 and 10 bits), their histograms added up over distributed shared
// memory, find the key of the last unit that stays.  Exact zeros, which a cache
// is full of, are counted by ballot and not by atomics on one bin.  A unit's place
// in the list follows from two counts before it, larger keys and equal ones (of
// which the first `ties` stay), taken per warp over its own run: no barrier while
// the list is written.
//
// 32 caches of 131k-262k tokens (48 MB of mass) take 19 us, 37 % of the copy
// bandwidth; a cache of 4099 tokens 5 us, which is the chain of rounds and their
// barriers.
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

struct EvictCtrl {
  uint32_t hist[3][kEvBins];
  uint32_t merged[kEvBins];
  uint32_t warp_tot[kEvWarps], gt[kEvWarps], eq[kEvWarps];
  uint32_t gt_all, eq_all, above;
  int32_t bin, bad;
};
constexpr size_t kEvKeysOff = (sizeof(EvictCtrl) + 15) / 16 * 16;

// Keys of the (up to) four tokens from unit u0's first on: four units of one
// token, or one unit of four.
template <int UNIT>
__device__ __forceinline__ void unit_keys(const float *m, int64_t cols, int32_t nkv, int64_t t, uint32_t (&key)[4 / UNIT],
                                          bool (&bad)[4 / UNIT]) {
  float4 s = *reinterpret_cast<const float4 *>(m + t);
  for (int h = 1; h < nkv; ++h) {
    const float4 x = *reinterpret_cast<const float4 *>(m + h * cols + t);
    s.x = __fadd_rn(s.x, x.x);
    s.y = __fadd_rn(s.y, x.y);
    s.z = __fadd_rn(s.z, x.z);
    s.w = __fadd_rn(s.w, x.w);
  }
  if constexpr (UNIT == 4) {
    const float f = __fadd_rn(__fadd_rn(__fadd_rn(s.x, s.y), s.z), s.w);
    key[0] = order_key(f);
    bad[0] = !isfinite(f);
  } else {
    key[0] = order_key(s.x);
    key[1] = order_key(s.y);
    key[2] = order_key(s.z);
    key[3] = order_key(s.w);
    bad[0] = !isfinite(s.x);
    bad[1] = !isfinite(s.y);
    bad[2] = !isfinite(s.z);
    bad[3] = !isfinite(s.w);
  }
}

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
  // this CTA's units [u0, u1): a multiple of 1024, so that a warp's run is one of 32
  const int32_t seg = ((units + ctas - 1) / ctas + 1023) & ~1023;
  const int32_t u0 = min((int64_t)units, (int64_t)rank * seg), u1 = min((int64_t)units, (int64_t)u0 + seg);
  const int32_t lo = a.n_first / UNIT, hi = units - a.n_last / UNIT;  // units in [lo, hi) compete
  const float *m = a.mass + (int64_t)s * a.nkv * a.mass_cols;
  constexpr int kPer = 4 / UNIT;  // units per load
  __syncthreads();

  // ---- round 0 while the mass is read: keys, their upper 11 bits, and what is not finite
  const int32_t loads = (u1 - u0 + kPer - 1) / kPer;
  uint32_t zeros = 0;
  bool any_bad = false;
#pragma unroll 4
  for (int32_t i = tid; i < loads; i += kEvThreads) {
    uint32_t key[kPer];
    bool bad[kPer];
    unit_keys<UNIT>(m, a.mass_cols, a.nkv, ((int64_t)u0 + (int64_t)i * kPer) * UNIT, key, bad);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int32_t u = u0 + i * kPer + e;
      if (u >= u1) continue;
      any_bad |= bad[e];
      if (CACHED) keys[u - u0] = key[e];
      if (u < lo || u >= hi) continue;
      if (key[e] == kZeroKey) ++zeros;
      else atomicAdd(&C.hist[0][key[e] >> 21], 1u);
    }
  }
  for (int o = 16; o; o >>= 1) zeros += __shfl_xor_sync(0xffffffffu, zeros, o);
  if (lane == 0 && zeros) atomicAdd(&C.hist[0][kZeroKey >> 21], zeros);
  if (any_bad) C.bad = 1;

  auto key_at = [&](int32_t u) -> uint32_t {
    if (CACHED) return keys[u - u0];
    uint32_t key[kPer];
    bool bad[kPer];
    const int64_t t = (int64_t)u * UNIT;
    unit_keys<UNIT>(m, a.mass_cols, a.nkv, t & ~(int64_t)3, key, bad);
    if constexpr (UNIT == 4) return key[0];
    return (t & 3) == 0 ? key[0] : (t & 3) == 1 ? key[1] : (t & 3) == 2 ? key[2] : key[3];
  };

  // ---- the key of the last unit that stays: the cut-th largest of those that compete
  uint32_t need = (uint32_t)(keep - lo - (units - hi)), prefix = 0;
  const bool none = need == 0;  // the protected units fill the budget
#pragma unroll
  for (int round = 0; round < 3; ++round) {
    constexpr int kShift[3] = {21, 10, 0};
    const int bins = round == 2 ? 1024 : kEvBins;
    if (round > 0 && !none) {
      zeros = 0;
      for (int32_t u = max(u0, lo) + tid; u < min(u1, hi); u += kEvThreads) {
        const uint32_t k = key_at(u);
        if ((k >> (round == 1 ? 21 : 10)) != prefix) continue;
        if (k == kZeroKey) ++zeros;
        else atomicAdd(&C.hist[round][(k >> kShift[round]) & (uint32_t)(bins - 1)], 1u);
      }
      for (int o = 16; o; o >>= 1) zeros += __shfl_xor_sync(0xffffffffu, zeros, o);
      if (lane == 0 && zeros) atomicAdd(&C.hist[round][(kZeroKey >> kShift[round]) & (uint32_t)(bins - 1)], zeros);
    }
    all_sync();  // every CTA's histogram (and, in round 0, its verdict) is there
    if (round == 0) {
      bool bad = C.bad != 0;
      for (int32_t r = 0; ctas > 1 && r < ctas; ++r) bad |= *cluster.map_shared_rank(&C.bad, r) != 0;
      if (bad) {  // the same in every CTA, none of which may leave while it is read
        if (tid == 0 && rank == 0) report_error(a.status, kErrNonFinite, s);
        all_sync();
        return;
      }
    }
    if (none) break;
    if (ctas > 1) {
      uint32_t part[kEvBins / kEvThreads][kEvMaxCluster];  // every read of the others on its way at once
#pragma unroll
      for (int i = 0; i < bins / kEvThreads; ++i)
#pragma unroll
        for (int r = 0; r < kEvMaxCluster; ++r)
          part[i][r] = r < ctas ? cluster.map_shared_rank(&C.hist[round][0], r)[tid + i * kEvThreads] : 0u;
#pragma unroll
      for (int i = 0; i < bins / kEvThreads; ++i) {
        uint32_t sum = 0;
#pragma unroll
        for (int r = 0; r < kEvMaxCluster; ++r) sum += part[i][r];
        C.merged[tid + i * kEvThreads] = sum;
      }
      __syncthreads();
    }
    find_bin<kEvThreads>(ctas > 1 ? C.merged : C.hist[round], bins, need, C.warp_tot, &C.bin, &C.above);
    prefix = (prefix << (round == 2 ? 10 : 11)) | (uint32_t)C.bin;
    need -= C.above;
    __syncthreads();  // bin and merged are written again in the next round
  }
  const uint32_t cut = prefix, ties = none ? 0u : need;

  // ---- counts before each warp's run, then the list
  const int32_t run = seg / kEvWarps;
  const int32_t w0 = u0 + warp * run, w1 = min(u1, w0 + run);
  auto state = [&](int32_t u) -> int {  // 1: stays, 2: equal to the cut, 0: goes
    if (u >= w1) return 0;
    if (u < lo || u >= hi) return 1;
    if (none) return 0;
    const uint32_t k = key_at(u);
    return k > cut ? 1 : k == cut ? 2 : 0;
  };
  uint32_t gt = 0, eq = 0;
  for (int32_t b = w0; b < w1; b += 32) {
    const int st = state(b + lane);
    gt += __popc(__ballot_sync(0xffffffffu, st == 1));
    eq += __popc(__ballot_sync(0xffffffffu, st == 2));
  }
  if (lane == 0) {
    C.gt[warp] = gt;
    C.eq[warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  uint32_t gt_all = 0, eq_all = 0;
#pragma unroll
  for (int i = 0; i < kEvWarps; ++i) {
    gt += i < warp ? C.gt[i] : 0u;
    eq += i < warp ? C.eq[i] : 0u;
    gt_all += C.gt[i];
    eq_all += C.eq[i];
  }
  if (tid == 0) {
    C.gt_all = gt_all;
    C.eq_all = eq_all;
  }
  if (ctas > 1) {
    cluster.sync();
    for (int32_t r = 0; r < rank; ++r) {
      gt += *cluster.map_shared_rank(&C.gt_all, r);
      eq += *cluster.map_shared_rank(&C.eq_all, r);
    }
    cluster.sync();  // no CTA leaves while its counts are read
  }
  for (int32_t b = w0; b < w1; b += 32) {
    const int32_t u = b + lane;
    const int st = state(u);
    const uint32_t g = __ballot_sync(0xffffffffu, st == 1), q = __ballot_sync(0xffffffffu, st == 2);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t my_eq = eq + __popc(q & below);
    const uint32_t at = gt + __popc(g & below) + min(my_eq, ties);
    if (st == 1 || (st == 2 && my_eq < ties)) {
#pragma unroll
      for (int e = 0; e < UNIT; ++e) sel[(int64_t)at * UNIT + e] = u * UNIT + e;
    }
    gt += __popc(g);
    eq += __popc(q);
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
  while (ctas < kEvMaxCluster && (units / ctas > kEvMaxKeys - 1024 ||
                                  (units / ctas > 4096 && (int64_t)n_seqs * ctas * 2 <= (int64_t)device_sm_count())))
    ctas *= 2;
  const int32_t keys = ((units + ctas - 1) / ctas + 1023) & ~1023;
  if (a.unit == 4)
    return keys <= kEvMaxKeys ? launch_evict<4, true>(a, n_seqs, ctas, keys, stream)
                              : launch_evict<4, false>(a, n_seqs, ctas, keys, stream);
  return keys <= kEvMaxKeys ? launch_evict<1, true>(a, n_seqs, ctas, keys, stream)
                            : launch_evict<1, false>(a, n_seqs, ctas, keys, stream);
}

}  // namespace qsa
