// Kept tokens of a paged cache moved to the front, in place and in order.
//
// Token keep[j] of a sequence moves to token first + j: its K and V rows, its
// mass in each KV head, and (whole blocks) its pooled block key.  keep[j] >=
// first + j, so a token only moves towards the front.
//
// One CTA owns a narrow column slice of a sequence's rows and walks the list
// from the front in chunks, each chunk read whole before any of it is written:
// a later chunk's sources lie at or past its own first destination, so no
// write reaches a source that is still to be read, and the slices never meet.
#include "qsa_launch.h"
#include "qsa_paged.cuh"

namespace qsa {

namespace {

constexpr int kCoThreads = 256;
constexpr int kCoLoads = 8;  // in flight per thread

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

constexpr int kSliceVecs = 4;  // 64 bytes of a row

__global__ void __launch_bounds__(kCoThreads) compact_kernel(const CompactArgs a) {
  grid_dependency_sync();
  const int32_t s = blockIdx.y;
  int32_t slice = blockIdx.x;
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
  const int32_t row_slices = (a.width / 8 + kSliceVecs - 1) / kSliceVecs;
  if (slice < 2 * row_slices) {
    uint16_t *pool = slice < row_slices ? a.k_pool : a.v_pool;
    const int32_t v0 = (slice % row_slices) * kSliceVecs;
    const bool in = v0 + (int)(threadIdx.x % kSliceVecs) < a.width / 8;
    auto at = [&](int64_t sl) { return reinterpret_cast<uint4 *>(pool + sl * a.width) + v0; };
    move_slice<uint4, kSliceVecs>(
        n,
        [&](int32_t j) -> const uint4 * {
          const int32_t t = source(j);
          const int64_t x = t < 0 ? -1 : slot(t), y = slot(first + j);
          if (x < 0 || y < 0) {
            report_error(a.status, kErrTokenRange, s);
            return nullptr;
          }
          return in && x != y ? at(x) : nullptr;
        },
        [&](int32_t j) { return at(slot(first + j)); });
    return;
  }
  slice -= 2 * row_slices;
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
  auto key = [&](int64_t b) { return reinterpret_cast<uint4 *>(a.block_keys + (base + b) * kHeadDim) + slice * kSliceVecs; };
  move_slice<uint4, kSliceVecs>(
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

}  // namespace

cudaError_t launch_cache_compact(const CompactArgs &a, int32_t n_seqs, cudaStream_t stream) {
  const int32_t row_slices = (a.width / 8 + kSliceVecs - 1) / kSliceVecs;
  const dim3 grid((unsigned)(2 * row_slices + a.nkv + kHeadDim / 8 / kSliceVecs), (unsigned)n_seqs);
  return launch_dependent(compact_kernel, grid, dim3(kCoThreads), 0, stream, 1u, a);
}

}  // namespace qsa
