// Kept tokens of a paged cache moved to the front, in place and in order.
//
// Token keep[j] of a sequence moves to token first + j: its K and V rows, its
// mass in each KV head, and (whole blocks) its pooled block key.  keep[j] >=
// first + j, so a token only moves towards the front.
//
// One CTA owns a narrow column slice of a sequence's K and V rows and walks the
// list from the front in chunks of 32 KiB, up to five of them on their way into
// shared memory (cp.async) at a time.  A later chunk's sources lie at or past its
// own first destination, so only the loads of a chunk itself have to be over, in
// every thread, before it is stored: one barrier a chunk.  A thread stores what it
// loaded.  The slices never meet, and no row is moved twice.
//
// The bound is HBM: every moved byte is read and written once.  Pool rows are looked
// up once per token and CTA, ahead of the copies.
#include "qsa_launch.h"
#include "qsa_paged.cuh"
#include "qsa_tc_cache.cuh"

namespace qsa {

namespace {

constexpr int kCoThreads = 512;
constexpr int kCoLoads = 4;  // per thread and chunk

// Moves of one sequence's list: element (j, c) goes from src(j) to dst(j).
template <typename T, int VECS, typename Src, typename Dst>
__device__ __forceinline__ void move_slice(int32_t n, Src src, Dst dst) {
  constexpr int kChunk = kCoThreads * kCoLoads / VECS;
  const int c = threadIdx.x % VECS, j0 = threadIdx.x / VECS;
  for (int32_t b = 0; b < n; b += kChunk) {
    T x[kCoLoads];
    T *to[kCoLoads];
#pragma unroll
    for (int i = 0; i < kCoLoads; ++i) {
      const int32_t j = b + j0 + i * (kCoThreads / VECS);
      const T *from = j < n ? src(j) : nullptr;
      to[i] = from ? dst(j) : nullptr;
      if (from) x[i] = from[c];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCoLoads; ++i)
      if (to[i]) to[i][c] = x[i];
  }
}

constexpr int kKeyVecs = 4;  // 64 bytes of a block key per CTA

constexpr int kCoDepth = 5;                              // chunks in flight at most
constexpr uint32_t kCoChunk = kCoThreads * kCoLoads * 16;  // bytes of a chunk

// SV 16-byte vectors of each K row and of each V row per CTA.
template <int SV>
__global__ void __launch_bounds__(kCoThreads)
compact_kernel(const CompactArgs a, int32_t n_seqs, int32_t depth) {
  extern __shared__ __align__(16) uint8_t co_smem[];
  grid_dependency_sync();
  // every sequence's row slices first, then what is short: a CTA of those ahead of
  // a row slice would push it into a second wave
  const int32_t vecs = a.width / 8, row_slices = (vecs + SV - 1) / SV;
  const int32_t more = (int32_t)gridDim.x / n_seqs - row_slices, at = (int32_t)blockIdx.x - n_seqs * row_slices;
  const int32_t s = at < 0 ? (int32_t)blockIdx.x / row_slices : at / more;
  int32_t slice = at < 0 ? (int32_t)blockIdx.x % row_slices : row_slices + at % more;
  const int32_t n = a.n_keep[s], first = a.first ? a.first[s] : 0;
  if (n < 0 || n > a.max_keep || first < 0 || (int64_t)first + n > (int64_t)a.table_len * a.page.d ||
      (a.mass && (int64_t)first + n > a.mass_cols)) {
    if (threadIdx.x == 0 && slice == 0) report_error(a.status, kErrRowRange, s);
    return;
  }
  const int32_t *keep = a.keep + (int64_t)s * a.keep_cols;
  const int32_t *table = a.table + (int64_t)s * a.table_cols;
  const int64_t most = a.mass ? min((int64_t)a.mass_cols, (int64_t)a.table_len * a.page.d)
                              : (int64_t)a.table_len * a.page.d;
  auto slot = [&](int32_t t) -> int64_t {
    const int32_t pg = fast_div(a.page, t), phys = table[pg];
    if (phys < 0 || phys >= a.pool_pages) return -1;
    return (int64_t)phys * a.page.d + (t - pg * a.page.d);
  };
  auto source = [&](int32_t j) -> int32_t {  // keep[j], or -1 where it may not move
    const int32_t t = keep[j];
    return t < first + j || t >= most ? -1 : t;
  };
  if (slice < row_slices) {
    constexpr int kLanes = 2 * SV, kRowsAtOnce = kCoThreads / kLanes, kChunk = kRowsAtOnce * kCoLoads;
    const int c = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
    const int32_t v = slice * SV + c % SV;
    uint4 *pool = reinterpret_cast<uint4 *>(c < SV ? a.k_pool : a.v_pool) + v;
    const int32_t chunks = (n + kChunk - 1) / kChunk;
    // shared memory: depth chunks, then (source, destination) rows of depth + 2
    uint8_t *ring = co_smem + threadIdx.x * 16;
    int2 *rows = reinterpret_cast<int2 *>(co_smem + (size_t)depth * kCoChunk);
    // A token a thread: its number, the two pages, the rows.  Each step waits for the
    // reads of the one before it, so the steps of a chunk lie a chunk apart: a look-up
    // made in one go took 3 us of every chunk.
    struct Look {
      int32_t t, px, py;
    };
    auto token = [&](int32_t k) -> int32_t {  // -1: not moved
      const int32_t j = k * kChunk + (int32_t)threadIdx.x;
      return threadIdx.x < kChunk && j < n ? keep[j] : -1;
    };
    auto pages = [&](int32_t k, int32_t t) -> Look {
      const int32_t j = k * kChunk + (int32_t)threadIdx.x;
      Look l = {t, -1, -1};
      if (threadIdx.x < kChunk && j < n) {
        if (t >= first + j && t < most) l.px = table[fast_div(a.page, t)];
        l.py = table[fast_div(a.page, first + j)];
      }
      return l;
    };
    auto put = [&](int32_t k, const Look &l) {
      const int32_t j = k * kChunk + (int32_t)threadIdx.x;
      if (threadIdx.x >= kChunk || k >= chunks) return;
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
      rows[(k % (depth + 2)) * kChunk + threadIdx.x] = row;
    };
    auto issue = [&](int32_t k) {  // chunk k into its place of the ring
      if (k < chunks && v < vecs) {
#pragma unroll
        for (int i = 0; i < kCoLoads; ++i) {
          const int32_t from = rows[(k % (depth + 2)) * kChunk + r0 + i * kRowsAtOnce].x;
          if (from >= 0)
            cp_async16(sm32(ring + (size_t)(k % depth) * kCoChunk + i * kCoThreads * 16), pool + (int64_t)from * vecs, 16u);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int32_t ts[kCoDepth + 1];
    Look ls[kCoDepth + 1];
#pragma unroll
    for (int k = 0; k <= kCoDepth; ++k) ts[k] = k <= depth ? token(k) : -1;
    int32_t far = token(depth + 1);
#pragma unroll
    for (int k = 0; k <= kCoDepth; ++k)
      if (k <= depth) ls[k] = pages(k, ts[k]);
    Look ahead = pages(depth + 1, far);
    far = token(depth + 2);
#pragma unroll
    for (int k = 0; k <= kCoDepth; ++k)
      if (k <= depth) put(k, ls[k]);
    __syncthreads();
    for (int32_t k = 0; k < depth; ++k) issue(k);
    for (int32_t k = 0; k < chunks; ++k) {
      switch (depth) {  // chunk k has landed, those behind it may be on their way
        case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
      }
      __syncthreads();
      if (v < vecs) {
#pragma unroll
        for (int i = 0; i < kCoLoads; ++i) {
          const int32_t to = rows[(k % (depth + 2)) * kChunk + r0 + i * kRowsAtOnce].y;
          if (to >= 0)
            pool[(int64_t)to * vecs] =
                *reinterpret_cast<const uint4 *>(ring + (size_t)(k % depth) * kCoChunk + i * kCoThreads * 16);
        }
      }
      issue(k + depth);
      put(k + depth + 1, ahead);
      ahead = pages(k + depth + 2, far);
      far = token(k + depth + 3);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  slice -= row_slices;
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

template <int SV>
cudaError_t launch_compact(const CompactArgs &a, int32_t n_seqs, cudaStream_t stream) {
  static PerDevice smem_attr;
  constexpr int kRows = kCoThreads / (2 * SV) * kCoLoads;  // tokens per chunk
  auto smem = [](int32_t depth) { return (size_t)depth * kCoChunk + (size_t)(depth + 2) * kRows * sizeof(int2); };
  const cudaError_t e = set_smem_once(smem_attr, compact_kernel<SV>, smem(kCoDepth));
  if (e != cudaSuccess) return e;
  const int32_t row_slices = (a.width / 8 + SV - 1) / SV;
  const int32_t keys = a.block_keys ? kHeadDim / 8 / kKeyVecs : 0;
  const int64_t grid = (int64_t)(row_slices + a.nkv + keys) * n_seqs;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  // short lists leave shared memory to more CTAs
  const int32_t chunks = (a.max_keep + kRows - 1) / kRows, depth = chunks < kCoDepth ? chunks : kCoDepth;
  return launch_dependent(compact_kernel<SV>, dim3((unsigned)grid), dim3(kCoThreads), smem(depth), stream, 1u, a, n_seqs,
                          depth);
}

}  // namespace

cudaError_t launch_cache_compact(const CompactArgs &a, int32_t n_seqs, cudaStream_t stream) {
  // the widest slice (128, 64 or 32 bytes of K and of V) that still gives most SMs one
  const int64_t vecs = (int64_t)a.width / 8 * n_seqs, want = (int64_t)device_sm_count() * 3 / 4;
  if (vecs >= want * 8) return launch_compact<8>(a, n_seqs, stream);
  if (vecs >= want * 4) return launch_compact<4>(a, n_seqs, stream);
  return launch_compact<2>(a, n_seqs, stream);
}

}  // namespace qsa
