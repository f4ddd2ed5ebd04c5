// The attention weight that cached tokens gather.
//
// For KV head g of a sequence, token t's mass becomes
//   carry * mass[t] + sum_r w_r sum_{h in g} exp(scale q_rh . k_t - lse_rh)
// over the drafted rows r that see t; a drafted token's mass starts at zero.
//
// One warp per (sequence, KV head, token): a lane holds head_dim / 32 dims of
// the key, every row's heads are reduced by shuffles and added in row order.
#include "qsa_launch.h"
#include "qsa_paged.cuh"

namespace qsa {

namespace {

constexpr int kMassWarps = 8;

template <int HD>
__global__ void __launch_bounds__(32 * kMassWarps) attn_mass_kernel(const MassArgs a) {
  constexpr int kE = HD / 32;
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t s = blockIdx.y, kvh = blockIdx.z;
  const SeqView v = view_seq(a.seqs, s);
  if (!v.ok || v.ctx + v.rows > a.mass_cols) {
    if (threadIdx.x == 0 && blockIdx.x == 0) report_error(a.status, kErrRowRange, s);
    return;
  }
  if (v.rows == 0) return;
  for (int32_t t = blockIdx.x * kMassWarps + warp; t < v.ctx + v.rows; t += gridDim.x * kMassWarps) {
    const int64_t slot = token_slot(a.seqs, s, t);
    if (slot < 0) {
      if (lane == 0) report_error(a.status, kErrTokenRange, s);
      continue;
    }
    float k[kE], sum = 0.f;
    for (int e = 0; e < kE; ++e) k[e] = bf16_to_f32(a.k_pool[(slot * a.nkv + kvh) * HD + lane * kE + e]);
    for (int32_t j = 0; j < v.rows; ++j) {
      const int64_t row = v.row0 + j;
      const uint32_t *mrow = a.seqs.mask ? a.seqs.mask + row * a.seqs.mask_words : nullptr;
      if (t >= v.ctx && !sees_draft(mrow, j, t - v.ctx)) continue;
      const float w = a.weight ? a.weight[row] : 1.f;
      if (w == 0.f) continue;
      for (int32_t h = kvh * a.group; h < (kvh + 1) * a.group; ++h) {
        const uint16_t *q = a.q + row * a.q_stride + (int64_t)h * HD + lane * kE;
        float d = 0.f;
        for (int e = 0; e < kE; ++e) d = fmaf(bf16_to_f32(q[e]), k[e], d);
        for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        const float lse = a.lse[row * a.nq + h];
        if (lse != -INFINITY) sum = fmaf(w, expf(d * a.scale - lse), sum);
      }
    }
    float *m = a.mass + ((int64_t)s * a.nkv + kvh) * a.mass_cols + t;
    if (lane == 0) *m = t < v.ctx && a.carry != 0.f ? fmaf(a.carry, *m, sum) : sum;
  }
}

}  // namespace

cudaError_t launch_attn_mass(const MassArgs &a, int32_t head_dim, cudaStream_t stream) {
  const dim3 grid(512, (unsigned)a.seqs.n_seqs, (unsigned)a.nkv);
  if (head_dim == 256)
    return launch_dependent(attn_mass_kernel<256>, grid, dim3(32 * kMassWarps), 0, stream, 1u, a);
  return launch_dependent(attn_mass_kernel<128>, grid, dim3(32 * kMassWarps), 0, stream, 1u, a);
}

}  // namespace qsa
