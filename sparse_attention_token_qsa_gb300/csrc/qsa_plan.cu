// The pages, rows and slots of a step.
//
// need_s = ceil((ctx_s + new_s) / page).  The pages [need_s, held_s) go on a stack of
// free ones, in the order of sequences and entries; the pages [held_s, need_s) come off it
// in that order, the i-th from place H - 1 - i of the stack's height H; row j of
// sequence s is token ctx_s + j, in page table[s][(ctx_s + j) / page].
//
// Whole numbers only, and little of them: three passes over the sequences' lengths and
// one over the rows, 12 bytes each.  What costs is the chain: lengths, sums over the
// sequences, the stack, the tables, the rows.  One CTA does a small step; of many sequences
// or rows a cluster of eight, whose CTAs all sum the lengths and share the pages to move, with a
// cluster barrier where one reads what another wrote; so the lengths,
// heights and tables may be updated in place.  Many rows are filled by a second launch: 1024
// sequences of up to 256 rows, 131k in all, take 15.0 us (32.8 by one cluster alone, whose CTAs
// each moved their own sequences' pages).  64 single rows take 6.2 us, a launch and the chain
// (7.7 with the warps' sums added up one by one and the rows' places fetched from L2).
#include "qsa_launch.h"

namespace qsa {

namespace {

constexpr int kPlThreads = 1024, kPlWarps = kPlThreads / 32, kPlCtas = 8, kFillThreads = 256;

struct PlanSeq {
  int32_t rows, back, take, held;
  bool ok;
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs &a, int32_t s) {
  PlanSeq p = {0, 0, 0, 0, true};
  if (s >= a.n_seqs) return p;
  const int32_t ctx = a.ctx_len[s], rows = a.new_rows[s];
  p.held = a.held[s];
  p.ok = ctx >= 0 && rows >= 0 && p.held >= 0 && p.held <= a.table_len &&
         (int64_t)ctx + rows <= (int64_t)a.table_len * a.page.d;
  if (!p.ok) return p;
  p.rows = rows;
  const int32_t kv = ctx + rows, need = kv > 0 ? fast_div(a.page, kv - 1) + 1 : 0;
  p.back = max(0, p.held - need);
  p.take = max(0, need - p.held);
  return p;
}

// How many of the 32 lanes' ascending values are <= x (each lane its own x).
__device__ __forceinline__ int lanes_upto(int64_t value, int64_t x) {
  int n = 0;
#pragma unroll
  for (int step = 16; step; step >>= 1)
    if (__shfl_sync(0xffffffffu, value, n + step - 1) <= x) n += step;
  if (__shfl_sync(0xffffffffu, value, n) <= x) ++n;  // (n <= 31 here)
  return n;
}

__device__ __forceinline__ void plan_barrier() {
  if (gridDim.x == 1) {
    __syncthreads();
    return;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sets a flag in the shared memory of every CTA of the cluster; plan_barrier shows it to them.
__device__ __forceinline__ void flag_all(int32_t &flag) {
  if (gridDim.x == 1) {
    flag = 1;
    return;
  }
  const uint32_t here = (uint32_t)__cvta_generic_to_shared(&flag);
  for (uint32_t r = 0; r < gridDim.x; ++r)
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.u32 [a], %2;\n\t}" ::"r"(here), "r"(r), "r"(1)
                 : "memory");
}

struct PlanSums {
  int64_t rows, back, take;
};

// Warp `at` of `warps` fills its run of the rows' places, 32 at a time; `base`: a sequence no
// later than theirs.  start(s): sequence s's first row, ctx(s): its cached tokens.
template <typename Start, typename Ctx>
__device__ __forceinline__ void fill_rows(const PlanArgs &a, int64_t at, int64_t warps, int64_t rows, int lane, Start &&start, Ctx &&ctx) {
  const int64_t per = (((int64_t)a.max_rows + warps - 1) / warps + 31) / 32 * 32;
  const int64_t r0 = at * per, r1 = min((int64_t)a.max_rows, r0 + per);
  int32_t base = 0;
  if (r0 < rows) {  // the last sequence that starts at or before r0
    int32_t hi = a.n_seqs;
    while (hi - base > 1) {
      const int32_t step = (hi - base + 31) / 32, probe = base + lane * step;
      const uint32_t hit = __ballot_sync(0xffffffffu, probe < hi && start(probe) <= r0);
      base += (31 - __clz((int)hit)) * step;
      hi = min(hi, base + step);
    }
  }
  for (int64_t i0 = r0; i0 < r1; i0 += 32) {
    const int64_t r = i0 + lane;
    int32_t seq = -1;
    bool open = r < rows;
    while (__any_sync(0xffffffffu, open)) {
      const int64_t end = start(min(base + 1 + lane, a.n_seqs));
      const int n = lanes_upto(end, r);
      if (open && n < 32) {
        seq = base + n;
        open = false;
      }
      if (__any_sync(0xffffffffu, open)) base += 32;
    }
    if (i0 < rows) base = max(base, __reduce_max_sync(0xffffffffu, seq));
    if (r >= r1) continue;
    int32_t slot = -1, t = 0;
    if (seq >= 0) {
      t = ctx(seq) + (int32_t)(r - start(seq));
      const int32_t pg = fast_div(a.page, t), page = __ldcg(a.table + (int64_t)seq * a.table_cols + pg);
      if (page >= 0 && page < a.pool_pages) slot = page * a.page.d + (t - pg * a.page.d);
      else report_error(a.status, kErrTokenRange, seq);
    }
    a.slot[r] = slot;
    if (a.pos) a.pos[r] = t;
    if (a.row_seq) a.row_seq[r] = seq;
  }
}

__global__ void __launch_bounds__(kPlThreads) page_plan_kernel(const PlanArgs a, bool fill) {
  __shared__ int64_t scan[3][kPlWarps];
  // Up to as many sequences as threads: their first rows and contexts, which the rows
  // would else fetch in three trips to L2, one after another.
  __shared__ int32_t starts[kPlThreads + 1], contexts[kPlThreads];
  __shared__ int32_t spoiled;  // a page that is given back is none of the pool's
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = blockIdx.x, ranks = gridDim.x;  // the grid is one cluster
  if (tid == 0) spoiled = 0;
  // (met before another CTA's flag may be set)
  if (ranks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  grid_dependency_sync();

  // this thread's sequence of a chunk, and the sums before it; adds the chunk to `before`
  auto chunk = [&](int32_t s, PlanSeq &p, PlanSums &before) -> PlanSums {
    p = plan_seq(a, s);
    const int64_t r = warp_scan(p.rows, lane), b = warp_scan(p.back, lane), t = warp_scan(p.take, lane);
    __syncthreads();
    if (lane == 31) {
      scan[0][warp] = r;
      scan[1][warp] = b;
      scan[2][warp] = t;
    }
    __syncthreads();
    // the warps' sums, a lane a warp
    auto place = [&](const int64_t *sums, int64_t incl, int64_t &all) -> int64_t {
      const int64_t own = sums[lane], upto = warp_scan(own, lane), first = all + __shfl_sync(0xffffffffu, upto - own, warp);
      all += __shfl_sync(0xffffffffu, upto, 31);
      return first + incl;
    };
    PlanSums at;
    at.rows = place(scan[0], r - p.rows, before.rows);
    at.back = place(scan[1], b - p.back, before.back);
    at.take = place(scan[2], t - p.take, before.take);
    return at;
  };

  const int64_t free0 = *a.n_free;  // (on its way beside the lengths)
  PlanSums all = {0, 0, 0};
  PlanSeq p;
  PlanSums at = {0, 0, 0};
  for (int32_t s0 = 0; s0 < a.n_seqs; s0 += kPlThreads) {
    at = chunk(s0 + tid, p, all);
    if (rank == 0 && !p.ok) report_error(a.status, kErrRowRange, s0 + tid);
  }
  const bool one_chunk = a.n_seqs <= kPlThreads;  // p and at stay good
  const int64_t height = free0 + all.back;
  const bool stack_ok = free0 >= 0 && height <= a.pool_pages, rows_ok = all.rows <= a.max_rows;
  bool ok = stack_ok && rows_ok && all.take <= height;
  if (one_chunk && ok) {  // (met by the barriers before the rows)
    if (tid < a.n_seqs) {
      starts[tid] = (int32_t)at.rows;
      contexts[tid] = a.ctx_len[tid];
    }
    if (tid == 0) starts[a.n_seqs] = (int32_t)all.rows;
  }

  // The items of this warp's sequences, shared with the same warp of the other CTAs, which has
  // the same sequences: from(s, i, k) reads the i-th of sequence s's, the k-th of all, and
  // to(s, i, k, page) puts it in its place.  Four at once: each is a trip to L2.  True where a
  // page of this thread's is none of the pool's.
  auto each = [&](int32_t s, int32_t count, int64_t first, auto &&from, auto &&to) -> bool {
    bool bad = false;
    const int64_t incl = warp_scan(count, lane), total = __shfl_sync(0xffffffffu, incl, 31);
    const int64_t base = __shfl_sync(0xffffffffu, first, 0);
    constexpr int kAtOnce = 4;
    for (int64_t i0 = 32 * (int64_t)rank; i0 < total; i0 += 32 * kAtOnce * (int64_t)ranks) {
      int32_t seq[kAtOnce], at[kAtOnce], page[kAtOnce];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int64_t i = i0 + 32 * (int64_t)ranks * e + lane;
        const int src = min(lanes_upto(incl, i), 31);
        at[e] = (int32_t)(i - __shfl_sync(0xffffffffu, incl - count, src));
        seq[e] = __shfl_sync(0xffffffffu, s, src);
        if (i < total) page[e] = from(seq[e], at[e], base + i);
      }
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int64_t i = i0 + 32 * (int64_t)ranks * e + lane;
        if (i >= total) continue;
        if (page[e] < 0 || page[e] >= a.pool_pages) {
          report_error(a.status, kErrTokenRange, seq[e]);
          bad = true;
        }
        to(seq[e], at[e], base + i, page[e]);
      }
    }
    return bad;
  };

  if (ranks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (ok && all.back > 0) {
    PlanSums sums = {0, 0, 0};
    bool bad = false;
    for (int32_t s0 = 0; s0 < a.n_seqs; s0 += kPlThreads) {
      if (!one_chunk) at = chunk(s0 + tid, p, sums);
      bad |= each(s0 + tid, p.back, at.back,
                  [&](int32_t s, int32_t i, int64_t) -> int32_t {
                    const int32_t kv = a.ctx_len[s] + a.new_rows[s];
                    return a.table[(int64_t)s * a.table_cols + (kv > 0 ? fast_div(a.page, kv - 1) + 1 : 0) + i];
                  },
                  [&](int32_t, int32_t, int64_t k, int32_t page) { a.free_pages[free0 + k] = page; });
    }
    if (bad) flag_all(spoiled);
    plan_barrier();
    // The stack would hand the page to another sequence: nothing is planned (what was put
    // past the stack's height is not on it).
    ok = *static_cast<volatile int32_t *>(&spoiled) == 0;
  }
  {
    PlanSums sums = {0, 0, 0};
    for (int32_t s0 = 0; s0 < a.n_seqs; s0 += kPlThreads) {
      const int32_t s = s0 + tid;
      if (!one_chunk) at = chunk(s, p, sums);
      if (rank == 0 && s < a.n_seqs) {
        a.row_start[s] = ok ? (int32_t)at.rows : 0;
        if (s == a.n_seqs - 1) a.row_start[s + 1] = ok ? (int32_t)all.rows : 0;
        if (!ok) {
          if (!stack_ok) {
            if (s == 0) report_error(a.status, kErrTokenRange, 0);
          } else if (!rows_ok) {
            if (at.rows <= a.max_rows && at.rows + p.rows > a.max_rows) report_error(a.status, kErrRowRange, s);
          } else if (at.take <= height && at.take + p.take > height) {
            report_error(a.status, kErrNoPages, s);
          }
        }
      }
      if (!ok) continue;
      each(s, p.take, at.take, [&](int32_t, int32_t, int64_t k) -> int32_t { return __ldcg(a.free_pages + (height - 1 - k)); },
           [&](int32_t seq, int32_t i, int64_t, int32_t page) { a.table[(int64_t)seq * a.table_cols + a.held[seq] + i] = page; });
    }
  }
  plan_barrier();

  // everyone has read the lengths and heights: they may be written in place
  for (int64_t s = (int64_t)rank * kPlThreads + tid; s < a.n_seqs; s += (int64_t)ranks * kPlThreads) {
    const PlanSeq q = plan_seq(a, (int32_t)s);
    a.held_out[s] = !ok || !q.ok ? a.held[s] : q.held - q.back + q.take;
  }
  if (rank == 0 && tid == 0) *a.n_free_out = ok ? (int32_t)(height - all.take) : (int32_t)free0;

  if (!fill) return;
  const int64_t mine = (int64_t)rank * kPlWarps + warp, warps = (int64_t)ranks * kPlWarps, rows = ok ? all.rows : 0;
  if (one_chunk) fill_rows(a, mine, warps, rows, lane, [&](int32_t s) { return starts[s]; }, [&](int32_t s) { return contexts[s]; });
  else fill_rows(a, mine, warps, rows, lane, [&](int32_t s) { return __ldcg(a.row_start + s); }, [&](int32_t s) { return a.ctx_len[s]; });
}

// The rows of a large step, by all SMs.
__global__ void __launch_bounds__(kFillThreads) plan_rows_kernel(const PlanArgs a) {
  grid_dependency_sync();
  const int64_t warps = (int64_t)gridDim.x * (kFillThreads / 32);
  fill_rows(a, (int64_t)blockIdx.x * (kFillThreads / 32) + (threadIdx.x >> 5), warps, a.row_start[a.n_seqs], threadIdx.x & 31,
            [&](int32_t s) { return __ldcg(a.row_start + s); }, [&](int32_t s) { return a.ctx_len[s]; });
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs &a, cudaStream_t stream) {
  const unsigned ctas = a.n_seqs > 256 || a.max_rows > 4096 ? kPlCtas : 1;
  // Beyond the cluster's reach the rows are a launch of their own.
  const bool fill = a.max_rows <= 8192;
  const cudaError_t e = launch_dependent(page_plan_kernel, dim3(ctas), dim3(kPlThreads), 0, stream, ctas, a, fill);
  if (e != cudaSuccess || fill) return e;
  const int64_t blocks = ((int64_t)a.max_rows + 4 * kFillThreads - 1) / (4 * kFillThreads), most = 4 * device_sm_count();
  return launch_dependent(plan_rows_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kFillThreads), 0, stream, 1u, a);
}

}  // namespace qsa
