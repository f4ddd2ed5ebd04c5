// Attention of drafted rows over a paged K/V cache.
//
// A sequence has ctx cached tokens and n drafted ones behind them (a tree laid
// out in an order where a parent comes first); drafted row j attends every
// context token and the drafted tokens its mask names:
//   s_t = scale q . k_t,  lse = ln sum_t exp(s_t),  out = sum_t exp(s_t - lse) v_t.
//
// One CTA of four warps per (row, query head).  A warp takes every fourth
// token: a lane holds head_dim / 32 dims of q and of the running sum, the dot
// is reduced by shuffles, and the running maximum and sum of the softmax are
// updated per token; the warps' states are joined once at the end.
#include "qsa_launch.h"
#include "qsa_paged.cuh"

namespace qsa {

namespace {

constexpr int kWarps = 4;

template <int HD>
__global__ void __launch_bounds__(32 * kWarps) tree_attn_kernel(const TreeArgs a) {
  constexpr int kE = HD / 32;
  __shared__ float acc_s[kWarps][HD], m_s[kWarps], l_s[kWarps];
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t row = blockIdx.x / a.nq, h = blockIdx.x % a.nq;
  const int32_t s = seq_of_row(a.seqs, row);
  const SeqView v = view_seq(a.seqs, s);
  if (!v.ok) {
    if (threadIdx.x == 0) report_error(a.status, kErrRowRange, s);
    return;
  }
  if (row < v.row0 || row >= v.row0 + v.rows) return;
  const int32_t j = row - v.row0, kvh = h / a.group;
  const uint32_t *mrow = a.seqs.mask ? a.seqs.mask + (int64_t)row * a.seqs.mask_words : nullptr;
  float q[kE], acc[kE], m = -INFINITY, l = 0.f;
  for (int e = 0; e < kE; ++e) {
    q[e] = bf16_to_f32(a.q[(int64_t)row * a.q_stride + (int64_t)h * HD + lane * kE + e]);
    acc[e] = 0.f;
  }
  for (int32_t t = warp; t < v.ctx + v.rows; t += kWarps) {
    if (t >= v.ctx && !sees_draft(mrow, j, t - v.ctx)) continue;
    const int64_t slot = token_slot(a.seqs, s, t);
    if (slot < 0) {
      if (lane == 0) report_error(a.status, kErrTokenRange, s);
      continue;
    }
    const int64_t at = (slot * a.nkv + kvh) * HD + lane * kE;
    float d = 0.f;
    for (int e = 0; e < kE; ++e) d = fmaf(q[e], bf16_to_f32(a.k_pool[at + e]), d);
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    const float x = d * a.scale_log2;
    const float m1 = fmaxf(m, x), use = m1 == -INFINITY ? 0.f : m1;
    const float keep = exp2f(m - use), p = exp2f(x - use);
    m = m1;
    l = fmaf(l, keep, p);
    for (int e = 0; e < kE; ++e) acc[e] = fmaf(acc[e], keep, p * bf16_to_f32(a.v_pool[at + e]));
  }
  for (int e = 0; e < kE; ++e) acc_s[warp][lane * kE + e] = acc[e];
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, total = 0.f, w[kWarps];
  for (int i = 0; i < kWarps; ++i) top = fmaxf(top, m_s[i]);
  for (int i = 0; i < kWarps; ++i) {
    w[i] = exp2f(m_s[i] - (top == -INFINITY ? 0.f : top));
    total = fmaf(l_s[i], w[i], total);
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  for (int d = threadIdx.x; d < HD; d += 32 * kWarps) {
    float o = 0.f;
    for (int i = 0; i < kWarps; ++i) o = fmaf(acc_s[i][d], w[i], o);
    a.out[(int64_t)row * a.out_stride + (int64_t)h * HD + d] = (uint16_t)f32_to_bf16(o * inv);
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[(int64_t)row * a.nq + h] = total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
}

}  // namespace

int64_t tree_workspace_bytes(int32_t n_seqs, int32_t n_rows, int32_t group, int32_t head_dim) {
  constexpr int64_t kCtas = 160;
  const int64_t rows = (int64_t)n_rows * group < 128 ? (int64_t)n_rows * group : 128;
  return ((int64_t)(n_seqs + 1) * 8 + 255) / 256 * 256 + kCtas * 2 * rows * (head_dim + 2) * 4;
}

cudaError_t launch_tree_attn(const TreeArgs &a, int32_t head_dim, cudaStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.seqs.n_rows * a.nq));
  if (head_dim == 256)
    return launch_dependent(tree_attn_kernel<256>, grid, dim3(32 * kWarps), 0, stream, 1u, a);
  return launch_dependent(tree_attn_kernel<128>, grid, dim3(32 * kWarps), 0, stream, 1u, a);
}

}  // namespace qsa
