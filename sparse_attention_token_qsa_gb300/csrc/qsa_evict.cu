// The tokens a shortened cache keeps: the units (1 or 4 tokens) of the largest
// accumulated attention mass, the first and the last ones always among them.
//
// A unit's mass is the f32 sum of its tokens' in token order, a token's the
// f32 sum over the KV heads in head order; units are ordered by mass
// descending, then index ascending (-0 equals +0).
//
// One CTA per sequence: four passes of eight bits over monotonic 32-bit keys
// find the key of the last unit that stays, and one more pass writes the
// kept tokens in order, units equal to that key taken from the front.
#include "qsa_launch.h"
#include "qsa_paged.cuh"

namespace qsa {

namespace {

constexpr int kEvThreads = 1024;

__device__ __forceinline__ uint32_t mass_key(float f) {
  const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float unit_mass(const EvictArgs &a, int32_t s, int32_t u) {
  const float *m = a.mass + (int64_t)s * a.nkv * a.mass_cols;
  float sum = 0.f;
  for (int e = 0; e < a.unit; ++e) {
    const int64_t t = (int64_t)u * a.unit + e;
    float tok = m[t];
    for (int h = 1; h < a.nkv; ++h) tok = __fadd_rn(tok, m[h * a.mass_cols + t]);
    sum = e == 0 ? tok : __fadd_rn(sum, tok);
  }
  return sum;
}

__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *tot, uint32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = x;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) tot[warp] = incl;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
  for (int i = 0; i < kEvThreads / 32; ++i) {
    before += i < warp ? tot[i] : 0u;
    total += tot[i];
  }
  return before + incl - x;
}

__global__ void __launch_bounds__(kEvThreads) evict_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[256], tot[kEvThreads / 32], pick[2];
  __shared__ int bad;
  grid_dependency_sync();
  const int tid = threadIdx.x;
  const int32_t s = blockIdx.x;
  const int32_t len = a.length[s];
  if (len < 0 || len > a.tokens) {
    if (tid == 0) report_error(a.status, kErrRowRange, s);
    return;
  }
  const int32_t units = len / a.unit, keep = a.keep / a.unit;
  int32_t *sel = a.sel + (int64_t)s * a.sel_cols;
  if (units <= keep) {
    for (int32_t t = tid; t < len; t += kEvThreads) sel[t] = t;
    if (tid == 0) a.n_sel[s] = len;
    return;
  }
  const int32_t lo = a.n_first / a.unit, hi = units - a.n_last / a.unit;
  if (tid == 0) bad = 0;
  __syncthreads();
  for (int32_t u = tid; u < units; u += kEvThreads)
    if (!isfinite(unit_mass(a, s, u))) bad = 1;
  __syncthreads();
  if (bad) {
    if (tid == 0) report_error(a.status, kErrNonFinite, s);
    return;
  }
  uint32_t prefix = 0, want = keep - lo - (units - hi), ties = 0;  // units to take in (lo, hi)
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kEvThreads) hist[i] = 0;
      __syncthreads();
      for (int32_t u = lo + tid; u < hi; u += kEvThreads) {
        const uint32_t k = mass_key(unit_mass(a, s, u));
        if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t above = 0;
        int b = 255;
        while (above + hist[b] < want) above += hist[b--];
        pick[0] = (uint32_t)b;
        pick[1] = above;
      }
      __syncthreads();
      prefix = (prefix << 8) | pick[0];
      want -= pick[1];
      __syncthreads();
    }
    ties = want;
  }
  const bool none = keep == lo + units - hi;
  uint32_t base = 0, tied = 0;
  for (int32_t u0 = 0; u0 < units; u0 += kEvThreads) {
    const int32_t u = u0 + tid;
    uint32_t eq = 0, in = 0, total;
    if (u < units) {
      if (u < lo || u >= hi) in = 1;
      else if (!none) {
        const uint32_t k = mass_key(unit_mass(a, s, u));
        in = k > prefix;
        eq = k == prefix;
      }
    }
    const uint32_t r = tied + block_scan(eq, tot, total);
    tied += total;
    if (eq && r < ties) in = 1;
    const uint32_t at = base + block_scan(in, tot, total);
    base += total;
    if (in)
      for (int e = 0; e < a.unit; ++e) sel[(int64_t)at * a.unit + e] = u * a.unit + e;
  }
  for (int32_t t = units * a.unit + tid; t < len; t += kEvThreads) sel[(int64_t)keep * a.unit + t - units * a.unit] = t;
  if (tid == 0) a.n_sel[s] = a.keep + len - units * a.unit;
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs &a, int32_t n_seqs, cudaStream_t stream) {
  return launch_dependent(evict_kernel, dim3((unsigned)n_seqs), dim3(kEvThreads), 0, stream, 1u, a);
}

}  // namespace qsa
