// Attention over a paged cache held in 8 bits, with a scale for each block of tokens and
// head, and with a window over the tokens that a row looks back at.
//
// One CTA a row and KV head: its warps take the row's tokens in turn, a warp's lanes the
// dims, with the running maximum and sum of a softmax; the warps' parts are joined in
// shared memory.
#include "qsa_launch.h"
#include "qsa_tc_cache.cuh"

namespace qsa {

namespace {

constexpr int kC8Warps = 8, kC8Threads = 32 * kC8Warps;

__device__ __forceinline__ float of_e4m3(uint32_t byte) {
  uint32_t f;
  float x;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)byte));
  asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(x) : "r"(f));
  return x;
}

template <int HD>
__global__ void __launch_bounds__(kC8Threads) cache8_simple_kernel(const Cache8Args a) {
  constexpr int kDims = HD / 32;
  __shared__ float part[kC8Warps][HD], tops[kC8Warps], sums[kC8Warps];
  __shared__ int32_t found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t row = blockIdx.x, kvh = blockIdx.y;
  grid_dependency_sync();
  if (tid == 0) found = -1;
  __syncthreads();
  for (int32_t s = tid; s < a.seqs.n_seqs; s += kC8Threads) {
    const SeqView v = view_seq(a.seqs, s);
    if (!v.ok && row == 0 && kvh == 0) report_error(a.status, kErrRowRange, s);
    if (v.rows > 0 && row >= v.row0 && row < v.row0 + v.rows) found = s;
  }
  __syncthreads();
  const int32_t s = found;
  if (s < 0) return;
  const SeqView v = view_seq(a.seqs, s);
  const int32_t j = row - v.row0;
  const uint32_t *mrow = a.seqs.mask ? a.seqs.mask + (int64_t)row * a.seqs.mask_words : nullptr;
  int32_t at = v.ctx + j;
  if (mrow) {
    int32_t c = 0;
    for (int32_t k = 0; k < v.rows; ++k) c += sees_draft(mrow, j, k);
    at = v.ctx + max(0, c - 1);
  }
  const int32_t end = mrow ? v.ctx + v.rows : v.ctx + j + 1;
  for (int h = 0; h < a.group; ++h) {
    const int32_t head = kvh * a.group + h;
    float q[kDims], acc[kDims], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int d = 0; d < kDims; ++d) {
      q[d] = bf16_to_f32(a.q[(int64_t)row * a.q_stride + (int64_t)head * HD + lane * kDims + d]);
      acc[d] = 0.f;
    }
    for (int32_t t = warp; t < end; t += kC8Warps) {
      const bool drafted = t >= v.ctx;
      if (drafted && !sees_draft(mrow, j, t - v.ctx)) continue;
      if (a.window > 0 && t >= a.n_first && at - t >= a.window && !(drafted && mrow)) continue;
      const int64_t slot = token_slot(a.seqs, s, t);
      if (slot < 0) {
        if (lane == 0) report_error(a.status, kErrTokenRange, s);
        continue;
      }
      const int64_t block = (slot >> a.unit_log) * a.nkv + kvh, byte = (slot * a.nkv + kvh) * HD + lane * kDims;
      const float ks = a.k_scale[block], vs = a.v_scale[block];
      if (!(ks >= 0.f && ks < INFINITY && vs >= 0.f && vs < INFINITY) && lane == 0) report_error(a.status, kErrNonFinite, s);
      float x = 0.f;
#pragma unroll
      for (int d = 0; d < kDims; ++d) x = fmaf(q[d], of_e4m3(a.k_pool[byte + d]), x);
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      x *= ks * a.scale_log2;
      const float now = fmaxf(top, x), use = now == -INFINITY ? 0.f : now, keep = ex2(top - use), p = ex2(x - use);
      top = now;
      sum = fmaf(sum, keep, p);
#pragma unroll
      for (int d = 0; d < kDims; ++d) acc[d] = fmaf(p * vs, of_e4m3(a.v_pool[byte + d]), acc[d] * keep);
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < kDims; ++d) part[warp][lane * kDims + d] = acc[d];
    if (lane == 0) {
      tops[warp] = top;
      sums[warp] = sum;
    }
    __syncthreads();
    float most = -INFINITY, all = 0.f;
    for (int w = 0; w < kC8Warps; ++w) most = fmaxf(most, tops[w]);
    const float use = most == -INFINITY ? 0.f : most;
    for (int w = 0; w < kC8Warps; ++w) all = fmaf(sums[w], ex2(tops[w] - use), all);
    if (tid < HD) {
      float o = 0.f;
      for (int w = 0; w < kC8Warps; ++w) o = fmaf(part[w][tid], ex2(tops[w] - use), o);
      a.out[(int64_t)row * a.out_stride + (int64_t)head * HD + tid] = (uint16_t)f32_to_bf16(all == 0.f ? 0.f : o / all);
    }
    if (tid == 0 && a.lse)
      a.lse[(int64_t)row * a.nq + head] = all == 0.f ? -INFINITY : (most + log2f(all)) * 0.6931471805599453f;
  }
}

}  // namespace

int64_t cache8_workspace_bytes(int32_t n_seqs, int32_t n_rows, int32_t group, int32_t head_dim) {
  return 256 + (int64_t)n_seqs * 8 + (int64_t)n_rows * 4 + 0 * group * head_dim;
}

cudaError_t launch_cache8_attn(const Cache8Args &a, int32_t head_dim, cudaStream_t stream) {
  const dim3 grid((unsigned)a.seqs.n_rows, (unsigned)a.nkv);
  return launch_dependent(head_dim == 256 ? cache8_simple_kernel<256> : cache8_simple_kernel<128>, grid, dim3(kC8Threads), 0,
                          stream, 1u, a);
}

}  // namespace qsa
