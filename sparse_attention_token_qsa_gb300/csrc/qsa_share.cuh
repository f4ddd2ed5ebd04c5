// A launch's work as one list that runs through its sequences: each CTA takes an
// equal, contiguous share of it, so ragged batches balance.
#pragma once

#include "qsa_paged.cuh"

namespace qsa {

struct ShareScratch {
  int64_t scan[32], found_off;
  int32_t found_seq;
};

struct FoundShare {
  TileShare share;
  int64_t total, off;  // off: where the share begins in sequence seq's part of the list
  int32_t seq;
};

// count(s): what sequence s has in the list (0 for s >= n_seqs).  Every thread of the
// CTA (`threads` of them, whole warps, 1024 at most) calls it.
template <typename Count>
__device__ __forceinline__ FoundShare find_share(int32_t n_seqs, int threads, uint32_t sharers, uint32_t at, ShareScratch &m,
                                                 Count &&count) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
  FoundShare f;
  f.seq = n_seqs;
  f.off = 0;
  if (n_seqs <= 32) {  // a lane each, every warp for itself
    const int64_t c = count(lane), incl = warp_scan(c, lane), begin = incl - c;
    f.total = __shfl_sync(0xffffffffu, incl, 31);
    f.share = tile_share(f.total, sharers, at);
    const uint32_t hit =
        __ballot_sync(0xffffffffu, f.share.n > 0 && c > 0 && begin <= f.share.first && f.share.first < incl);
    if (hit != 0) {
      f.seq = __ffs(hit) - 1;
      f.off = f.share.first - __shfl_sync(0xffffffffu, begin, f.seq);
    }
    return f;
  }
  if (tid == 0) {
    m.found_seq = n_seqs;
    m.found_off = 0;
  }
  const bool one_chunk = n_seqs <= threads;
  f.total = 0;
  if (!one_chunk) {
    for (int32_t s = tid; s < n_seqs; s += threads) f.total += count(s);
    for (int o = 16; o; o >>= 1) f.total += __shfl_xor_sync(0xffffffffu, f.total, o);
    if (lane == 0) m.scan[warp] = f.total;
    __syncthreads();
    f.total = 0;
    for (int i = 0; i < warps; ++i) f.total += m.scan[i];
  }
  int64_t before = 0;
  for (int32_t s0 = 0; s0 < n_seqs; s0 += threads) {
    const int32_t s = s0 + tid;
    const int64_t c = s < n_seqs ? count(s) : 0, incl = warp_scan(c, lane);
    __syncthreads();
    if (lane == 31) m.scan[warp] = incl;
    __syncthreads();
    int64_t begin = before + incl - c;
    for (int i = 0; i < warps; ++i) {
      begin += i < warp ? m.scan[i] : 0;
      before += m.scan[i];
    }
    if (one_chunk) f.total = before;
    f.share = tile_share(f.total, sharers, at);
    if (f.share.n > 0 && c > 0 && begin <= f.share.first && f.share.first < begin + c) {
      m.found_seq = s;
      m.found_off = f.share.first - begin;
    }
    if (before > f.share.first) break;
  }
  __syncthreads();
  f.seq = m.found_seq;
  f.off = m.found_off;
  return f;
}

}  // namespace qsa
