// Kept tokens of a paged cache moved to the front, in place and in order.
//
// Token keep[j] of a sequence moves to token first + j: its K and V rows, its
// mass in each KV head, and (whole blocks) its pooled block key.  keep[j] >=
// first + j, so a token only moves towards the front.
//
// One CTA owns a narrow column slice of a sequence's K and V rows and walks the
// list from the front in chunks of 16 or 32 KiB, up to three of them on their way into
// shared memory (cp.async) at a time.  A later chunk's sources lie at or past its
// own first destination, and what a chunk's destinations hold is only read by chunks
// up to it: so a chunk's loads have to be over, in every thread, before it is
// stored, and nothing else: one barrier a chunk.  A thread stores what it loaded.
// The slices never meet, and no row is moved twice.
//
// The bound is HBM: every moved byte is read and written once.  Whole rows per CTA,
// a sequence's CTAs a cluster with a cluster barrier per round of chunks, took 274
// us for what 64-byte slices and no cluster do in 101 (16 caches of 16k-65k tokens
// cut to 8192; 81 % of the copy bandwidth).
#include "qsa_launch.h"
#include "qsa_paged.cuh"
#include "qsa_tc_cache.cuh"

namespace qsa {

namespace {

constexpr int kCoThreads = 512;
constexpr int kMoveLoads = 4;  // of what is short, per thread and chunk

// Moves of one sequence's list: element (j, c) goes from src(j) to dst(j).
template <typename T, int VECS, typename Src, typename Dst>
__device__ __forceinline__ void move_slice(int32_t n, Src src, Dst dst) {
  constexpr int kChunk = kCoThreads * kMoveLoads / VECS;
  const int c = threadIdx.x % VECS, j0 = threadIdx.x / VECS;
  for (int32_t b = 0; b < n; b += kChunk) {
    T x[kMoveLoads];
    T *to[kMoveLoads];
#pragma unroll
    for (int i = 0; i < kMoveLoads; ++i) {
      const int32_t j = b + j0 + i * (kCoThreads / VECS);
      const T *from = j < n ? src(j) : nullptr;
      to[i] = from ? dst(j) : nullptr;
      if (from) x[i] = from[c];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMoveLoads; ++i)
      if (to[i]) to[i][c] = x[i];
  }
}

constexpr int kKeyVecs = 4;  // 64 bytes of a block key per CTA

constexpr int kCoDepth = 3;  // chunks in flight at most

struct CompactGrid {
  int32_t n_seqs, slices;
  int32_t sv;                    // 16-byte vectors of a K (and of a V) row per slice
  int32_t tokens;                // per chunk, at most one a thread
  int32_t depth;                 // chunks in flight
};

// A chunk is LOADS vectors of 16 bytes a thread.
template <int LOADS>
__global__ void __launch_bounds__(kCoThreads)
compact_kernel(const CompactArgs a, const CompactGrid cfg, const FastDiv lanes) {
  constexpr uint32_t kCoChunk = kCoThreads * LOADS * 16;
  extern __shared__ __align__(16) uint8_t co_smem[];
  grid_dependency_sync();
  // every sequence's row slices first, then what is short: a CTA of those ahead of
  // a row slice would push it into a second wave
  const int32_t at = (int32_t)blockIdx.x - cfg.n_seqs * cfg.slices;
  const int32_t more = a.nkv + (a.block_keys ? kHeadDim / 8 / kKeyVecs : 0);
  const int32_t s = at < 0 ? (int32_t)blockIdx.x / cfg.slices : at / more;
  int32_t slice = at < 0 ? (int32_t)blockIdx.x % cfg.slices : at % more;
  const bool lead = at < 0 && slice == 0;
  const int32_t n = a.n_keep[s], first = a.first ? a.first[s] : 0;
  if (n < 0 || n > a.max_keep || first < 0 || (int64_t)first + n > (int64_t)a.table_len * a.page.d ||
      (a.mass && (int64_t)first + n > a.mass_cols)) {
    if (threadIdx.x == 0 && lead) report_error(a.status, kErrRowRange, s);
    return;
  }
  const int32_t *keep = a.keep + (int64_t)s * a.keep_cols;
  const int32_t *table = a.table + (int64_t)s * a.table_cols;
  const int64_t most = a.mass ? min((int64_t)a.mass_cols, (int64_t)a.table_len * a.page.d)
                              : (int64_t)a.table_len * a.page.d;
  auto source = [&](int32_t j) -> int32_t {  // keep[j], or -1 where it may not move
    const int32_t t = keep[j];
    return t < first + j || t >= most ? -1 : t;
  };
  if (at < 0) {
    const int32_t vecs = a.width / 8, per = cfg.tokens, depth = cfg.depth, chunks = (n + per - 1) / per;
    // this thread's vectors of a chunk: token, and column in the K or the V row
    int32_t tok[LOADS];
    uint4 *pool[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int32_t e = (int32_t)threadIdx.x + i * kCoThreads;
      tok[i] = fast_div(lanes, e);
      const int32_t c = e - tok[i] * lanes.d, v = slice * cfg.sv + (c < cfg.sv ? c : c - cfg.sv);
      if (tok[i] >= per || v >= vecs) tok[i] = -1;
      pool[i] = reinterpret_cast<uint4 *>(c < cfg.sv ? a.k_pool : a.v_pool) + v;
    }
    // Look-ups go by groups of `group` chunks, a token a thread: its number, the two
    // pages, the rows.  Each step waits for the reads of the one before it, so the
    // steps of a group lie a group apart (a chunk apart, every chunk took as long as a
    // read under load, 2.5 us).  Shared memory: depth chunks, then the (source,
    // destination) rows of a ring of groups: those of chunks k .. k + depth, one that
    // is being written, and one.
    const int32_t group = kCoThreads / per, groups_ahead = (group - 1 + depth) / group, slots = groups_ahead + 2;
    uint8_t *ring = co_smem + threadIdx.x * 16;
    int2 *rows = reinterpret_cast<int2 *>(co_smem + (size_t)depth * kCoChunk);
    const int32_t my_chunk = (int32_t)threadIdx.x / per, my_token = (int32_t)threadIdx.x - my_chunk * per;
    struct Look {
      int32_t t, px, py;
    };
    auto index = [&](int32_t q) -> int32_t {  // this thread's list entry of group q; n: none
      const int64_t k = (int64_t)q * group + my_chunk;
      return my_chunk < group && k < chunks ? min((int64_t)n, k * per + my_token) : n;
    };
    auto token = [&](int32_t q) -> int32_t {
      const int32_t j = index(q);
      return j < n ? keep[j] : -1;
    };
    auto pages = [&](int32_t q, int32_t t) -> Look {
      const int32_t j = index(q);
      Look l = {t, -1, -1};
      if (j < n) {
        if (t >= first + j && t < most) l.px = table[fast_div(a.page, t)];
        l.py = table[fast_div(a.page, first + j)];
      }
      return l;
    };
    auto put = [&](int32_t q, const Look &l) {  // -1: not moved
      const int32_t j = index(q);
      int2 row = make_int2(-1, -1);
      if (j < n) {
        if (l.px >= 0 && l.px < a.pool_pages && l.py >= 0 && l.py < a.pool_pages) {
          row.x = l.px * a.page.d + (l.t - fast_div(a.page, l.t) * a.page.d);
          row.y = l.py * a.page.d + (first + j - fast_div(a.page, first + j) * a.page.d);
          if (row.x == row.y) row.x = row.y = -1;
        } else if (slice == 0) {
          report_error(a.status, kErrTokenRange, s);
        }
      }
      rows[(q % slots) * kCoThreads + threadIdx.x] = row;
    };
    // a chunk's place in the ring of chunks, and its rows
    struct Place {
      int32_t k = 0, chunk = 0, in_group = 0, slot = 0;
    };
    auto step = [&](Place &p) {
      ++p.k;
      if (++p.chunk == depth) p.chunk = 0;
      if (++p.in_group == group) {
        p.in_group = 0;
        if (++p.slot == slots) p.slot = 0;
      }
    };
    auto issue = [&](Place &p) {  // a chunk into its place of the ring
      if (p.k < chunks) {
        const int2 *r = rows + p.slot * kCoThreads + p.in_group * per;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          const int32_t from = tok[i] >= 0 ? r[tok[i]].x : -1;
          if (from >= 0)
            cp_async16(sm32(ring + (size_t)p.chunk * kCoChunk + i * kCoThreads * 16), pool[i] + (int64_t)from * vecs, 16u);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      step(p);
    };
    int32_t ts[kCoDepth + 1];
    Look ls[kCoDepth + 1];
#pragma unroll
    for (int q = 0; q <= kCoDepth; ++q) ts[q] = q <= groups_ahead ? token(q) : -1;
    int32_t far = token(groups_ahead + 1);
#pragma unroll
    for (int q = 0; q <= kCoDepth; ++q)
      if (q <= groups_ahead) ls[q] = pages(q, ts[q]);
    Look ahead = pages(groups_ahead + 1, far);
    far = token(groups_ahead + 2);
#pragma unroll
    for (int q = 0; q <= kCoDepth; ++q)
      if (q <= groups_ahead) put(q, ls[q]);
    __syncthreads();
    Place in, out;
    for (int32_t k = 0; k < depth; ++k) issue(in);
    for (int32_t q = 0; out.k < chunks; step(out)) {
      switch (depth) {  // the chunk has landed, those behind it may be on their way
        case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
      }
      __syncthreads();
      const int2 *r = rows + out.slot * kCoThreads + out.in_group * per;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int32_t to = tok[i] >= 0 ? r[tok[i]].y : -1;
        if (to >= 0)
          pool[i][(int64_t)to * vecs] =
              *reinterpret_cast<const uint4 *>(ring + (size_t)out.chunk * kCoChunk + i * kCoThreads * 16);
      }
      issue(in);
      if (out.in_group == 0) {
        put(q + groups_ahead + 1, ahead);
        ahead = pages(q + groups_ahead + 2, far);
        far = token(q + groups_ahead + 3);
        ++q;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  if (slice < a.nkv) {
    if (a.mass == nullptr) return;
    float *m = a.mass + ((int64_t)s * a.nkv + slice) * a.mass_cols;
    move_slice<float, 1>(
        n,
        [&](int32_t j) -> const float * {
          const int32_t t = source(j);
          return t < 0 || t == first + j ? nullptr : m + t;
        },
        [&](int32_t j) { return m + first + j; });
    return;
  }
  slice -= a.nkv;  // 64 bytes of the block keys
  if (a.block_keys == nullptr) return;
  const int64_t base = a.key_base ? a.key_base[s] : 0;
  if (base < 0 || (first & 3) != 0) {
    if (threadIdx.x == 0 && slice == 0) report_error(a.status, kErrRowRange, s);
    return;
  }
  auto key = [&](int64_t b) { return reinterpret_cast<uint4 *>(a.block_keys + (base + b) * kHeadDim) + slice * kKeyVecs; };
  move_slice<uint4, kKeyVecs>(
      n / 4,
      [&](int32_t j) -> const uint4 * {
        const int32_t t = source(4 * j);
        if (t < 0 || (t & 3) != 0 || source(4 * j + 1) != t + 1 || source(4 * j + 2) != t + 2 || source(4 * j + 3) != t + 3) {
          report_error(a.status, kErrTokenRange, s);
          return nullptr;
        }
        return t == first + 4 * j ? nullptr : key(t >> 2);
      },
      [&](int32_t j) { return key((first >> 2) + j); });
}

template <int LOADS>
cudaError_t launch_compact(const CompactArgs &a, CompactGrid g, int64_t grid, cudaStream_t stream) {
  g.tokens = kCoThreads * LOADS / (2 * g.sv);
  if (g.tokens > kCoThreads) g.tokens = kCoThreads;  // a look-up per thread
  const int32_t chunks = (a.max_keep + g.tokens - 1) / g.tokens;
  g.depth = chunks < kCoDepth ? chunks : kCoDepth;  // short lists leave shared memory to more CTAs
  auto smem = [](int32_t depth, int32_t tokens) {
    const int32_t group = kCoThreads / tokens;
    return (size_t)depth * kCoThreads * LOADS * 16 +
           (size_t)((group - 1 + depth) / group + 2) * kCoThreads * sizeof(int2);
  };
  static PerDevice smem_attr;
  const cudaError_t e = set_smem_once(smem_attr, compact_kernel<LOADS>, smem(kCoDepth, kCoThreads));
  if (e != cudaSuccess) return e;
  return launch_dependent(compact_kernel<LOADS>, dim3((unsigned)grid), dim3(kCoThreads), smem(g.depth, g.tokens), stream, 1u,
                          a, g, make_fast_div(2 * g.sv));
}

}  // namespace

cudaError_t launch_cache_compact(const CompactArgs &a, int32_t n_seqs, cudaStream_t stream) {
  // Slices: as wide as still gives every SM two CTAs, between 64 bytes and 1 KiB of a row
  const int32_t vecs = a.width / 8;
  const int64_t least = (vecs + 63) / 64, finest = vecs < 4 ? 1 : vecs / 4;
  int64_t slices = 2 * device_sm_count() / n_seqs;
  slices = slices > finest ? finest : slices < least ? least : slices;
  CompactGrid g = {};
  g.n_seqs = n_seqs;
  g.sv = (int32_t)((vecs + slices - 1) / slices);
  g.slices = (vecs + g.sv - 1) / g.sv;
  const int32_t more = a.nkv + (a.block_keys ? kHeadDim / 8 / kKeyVecs : 0);
  const int64_t grid = (int64_t)n_seqs * (g.slices + more);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  // Chunks of 32 KiB where a CTA has an SM to itself (4 caches cut to 8192: 51 us, 57 with
  // 16 KiB), else of 16 (16 caches: 101 us, 110 with 32 KiB and 137 with 8).
  return (int64_t)n_seqs * g.slices <= device_sm_count() ? launch_compact<4>(a, g, grid, stream)
                                                         : launch_compact<2>(a, g, grid, stream);
}

}  // namespace qsa
