// The query and key heads of new tokens normed and rotated, K and V into the cache.
//
//   y = x / sqrt(mean(x^2) + eps) * (1 + w),  dims (i, i + 32), i < 32, turned by the
//   token's angle;  q: bf16;  K, V: bf16, or e4m3 of y / s with one scale s = 2^e for the
//   tokens of a block and a head, the least with max |y| <= 448 s.
//
// An item of work is (sequence, block of tokens, head): the block's new tokens of one
// query, key or value head, a CTA's at a time; a head's dims lie eight to a lane.
#include "qsa_launch.h"
#include "qsa_share.cuh"

namespace qsa {

namespace {

constexpr int kWrWarps = 8, kWrThreads = 32 * kWrWarps;

// s = 2^e, the least with amax <= 448 s = 1.75 * 2^8 s; 0 for 0.  amax is finite.
__device__ __forceinline__ float scale_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0.f ? 0.f : __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// Four values over s as e4m3 (nearest even, at most 448); what is not finite as NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;  // x + 0 x: an infinity becomes NaN, which the conversion keeps
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(fmaf(b, 0.f, b)), "f"(fmaf(a, 0.f, a)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(fmaf(d, 0.f, d)), "f"(fmaf(c, 0.f, c)));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

__device__ __forceinline__ float over(float x, float s) { return s > 0.f ? __fdiv_rn(x, s) : x * 0.f; }

// Eight values of e4m3 as f32.
__device__ __forceinline__ void unpack_e4m3(const uint2 &w, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t h = (uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
    uint32_t f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(h));
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
        : "r"(f));
  }
}

// The head of one token, lane g of its kLanes holding dims 8g to 8g + 7: normed (w not
// nullptr) and turned by the angle of position `at` (< 0: not turned).
template <int HD>
__device__ __forceinline__ void prepare_head(float (&x)[8], const uint16_t *w, float eps, const uint16_t *cos_t,
                                             const uint16_t *sin_t, int32_t at, int g) {
  if (w != nullptr) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
    for (int o = HD / 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = __frcp_rn(__fsqrt_rn(fmaf(sum, 1.f / HD, eps)));
    float f[8];
    unpack8(ldg_v4(w + 8 * g), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (1.f + f[i]);
  }
  float other[8];  // of the pair: 32 dims are four lanes away
#pragma unroll
  for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(0xffffffffu, x[i], 4);
  if (at >= 0 && g < 8) {
    float c[8], s[8];
    unpack8(ldg_v4(cos_t + (int64_t)at * kRot + 8 * g), c);
    unpack8(ldg_v4(sin_t + (int64_t)at * kRot + 8 * g), s);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], c[i], (g < 4 ? -other[i] : other[i]) * s[i]);
  }
}

template <int HD, bool EIGHT>
__global__ void __launch_bounds__(kWrThreads) qkv_write_kernel(const WriteArgs a) {
  __shared__ ShareScratch scratch;
  __shared__ float most[kWrWarps];
  __shared__ int32_t some[kWrWarps];
  constexpr int kLanes = HD / 8, kPer = 32 / kLanes;  // lanes of a head, tokens a warp takes at once
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane % kLanes;
  grid_dependency_sync();

  const int64_t heads = (int64_t)a.nq + 2 * a.nkv;
  const int ul = a.unit_log;
  auto blocks_of = [&](const SeqView &v) -> int32_t {
    return v.rows > 0 ? ((v.ctx + v.rows - 1) >> ul) - (v.ctx >> ul) + 1 : 0;
  };
  FoundShare f = find_share(a.seqs.n_seqs, kWrThreads, gridDim.x, blockIdx.x, scratch, [&](int32_t s) -> int64_t {
    if (s >= a.seqs.n_seqs) return 0;
    const SeqView v = view_seq(a.seqs, s);
    if (!v.ok && blockIdx.x == 0) report_error(a.status, kErrRowRange, s);
    return blocks_of(v) * heads;
  });
  SeqView v = {0, 0, 0, false};
  int64_t count = 0;
  if (f.share.n > 0) {
    v = view_seq(a.seqs, f.seq);
    count = blocks_of(v) * heads;
  }
  for (int64_t left = f.share.n, off = f.off; left > 0; --left, ++off) {
    while (off >= count) {
      off -= count;
      if (++f.seq >= a.seqs.n_seqs) return;
      v = view_seq(a.seqs, f.seq);
      count = blocks_of(v) * heads;
    }
    const int32_t nth = (int32_t)(off / heads), head = (int32_t)(off - nth * heads);
    const int32_t begin = ((v.ctx >> ul) + nth) << ul;
    const int32_t t0 = max(v.ctx, begin), t1 = (int32_t)min((int64_t)v.ctx + v.rows, (int64_t)begin + (1 << ul));
    // a token's position, or -1 where its row is left alone
    auto position = [&](int32_t t) -> int32_t {
      const int32_t at = a.pos ? a.pos[v.row0 + (t - v.ctx)] : t;
      const bool ok = at >= 0 && at < a.table_rows;
      if (!ok) report_error(a.status, kErrRowRange, f.seq);
      return ok ? at : -1;
    };
    const bool is_q = head < a.nq, is_k = !is_q && head < a.nq + a.nkv;
    const int32_t kvh = head - a.nq - (is_k ? 0 : a.nkv);
    auto read = [&](int32_t t) -> uint4 {
      const int64_t row = v.row0 + (t - v.ctx);
      const uint16_t *src = is_q ? a.q + row * a.q_stride + (int64_t)head * HD
                                 : (is_k ? a.k + row * a.k_stride : a.v + row * a.v_stride) + (int64_t)kvh * HD;
      return ldg_v4(src + 8 * g);
    };
    auto prepared = [&](int32_t t, int32_t at, float (&x)[8]) {  // every lane of the warp
      unpack8(read(t), x);
      if (is_q || is_k) prepare_head<HD>(x, is_q ? a.q_norm_w : a.k_norm_w, a.eps, a.cos_t, a.sin_t, at, g);
    };
    if (is_q || !EIGHT) {
      for (int32_t tw = t0 + warp * kPer; tw < t1; tw += kWrWarps * kPer) {
        const int32_t t = tw + lane / kLanes;
        const int32_t at = t < t1 ? position(t) : -1;
        uint4 o;
        if (is_q || is_k) {
          float x[8];
          prepared(min(t, t1 - 1), at, x);
          o = make_uint4(pack_bf16(f32_to_bf16(x[0]), f32_to_bf16(x[1])), pack_bf16(f32_to_bf16(x[2]), f32_to_bf16(x[3])),
                         pack_bf16(f32_to_bf16(x[4]), f32_to_bf16(x[5])), pack_bf16(f32_to_bf16(x[6]), f32_to_bf16(x[7])));
        } else {
          o = read(min(t, t1 - 1));
        }
        if (at < 0) continue;
        uint16_t *dst;
        if (is_q) {
          dst = a.q_out + (int64_t)(v.row0 + (t - v.ctx)) * a.out_stride + (int64_t)head * HD;
        } else {
          const int64_t slot = token_slot(a.seqs, f.seq, t);
          if (slot < 0) {
            report_error(a.status, kErrTokenRange, f.seq);
            continue;
          }
          dst = static_cast<uint16_t *>(is_k ? a.k_pool : a.v_pool) + (slot * a.nkv + kvh) * HD;
        }
        *reinterpret_cast<uint4 *>(dst + 8 * g) = o;
      }
      continue;
    }
    // a block's scale, then its values
    const int64_t slot0 = token_slot(a.seqs, f.seq, begin);  // a block lies in one page
    if (slot0 < 0) {
      if (tid == 0) report_error(a.status, kErrTokenRange, f.seq);
      continue;
    }
    float amax = 0.f;
    bool any = false;
    for (int32_t tw = t0 + warp * kPer; tw < t1; tw += kWrWarps * kPer) {
      const int32_t t = tw + lane / kLanes;
      const int32_t at = t < t1 ? position(t) : -1;
      float x[8];
      prepared(min(t, t1 - 1), at, x);
      if (at < 0) continue;
      any = true;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    any = __any_sync(0xffffffffu, any);
    __syncthreads();
    if (lane == 0) {
      most[warp] = amax;
      some[warp] = any;
    }
    __syncthreads();
    any = false;
    for (int i = 0; i < kWrWarps; ++i) {
      amax = fmaxf(amax, most[i]);
      any = any || some[i];
    }
    if (!any) continue;
    float *scale = (is_k ? a.k_scale : a.v_scale) + (slot0 >> ul) * a.nkv + kvh;
    uint8_t *pool = static_cast<uint8_t *>(is_k ? a.k_pool : a.v_pool) + (slot0 * a.nkv + kvh) * HD;
    const int64_t pitch = (int64_t)a.nkv * HD;
    const float old = t0 > begin ? *scale : 0.f, now = fmaxf(old, scale_of(amax));
    if (now > old) {
      for (int32_t t = begin + warp * kPer + lane / kLanes; t < t0; t += kWrWarps * kPer) {
        uint2 *at = reinterpret_cast<uint2 *>(pool + (t - begin) * pitch + 8 * g);
        float x[8];
        unpack_e4m3(*at, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = over(x[i] * old, now);
        *at = make_uint2(pack_e4m3(x[0], x[1], x[2], x[3]), pack_e4m3(x[4], x[5], x[6], x[7]));
      }
    }
    for (int32_t tw = t0 + warp * kPer; tw < t1; tw += kWrWarps * kPer) {
      const int32_t t = tw + lane / kLanes;
      const int32_t at = t < t1 ? position(t) : -1;
      float x[8];
      prepared(min(t, t1 - 1), at, x);
      if (at < 0) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = over(x[i], now);
      *reinterpret_cast<uint2 *>(pool + (t - begin) * pitch + 8 * g) =
          make_uint2(pack_e4m3(x[0], x[1], x[2], x[3]), pack_e4m3(x[4], x[5], x[6], x[7]));
    }
    __syncthreads();  // the old scale is read by everyone
    if (tid == 0) *scale = now;
  }
}

template <int HD>
cudaError_t launch_hd(const WriteArgs &a, cudaStream_t stream) {
  const int64_t blocks = ((int64_t)a.seqs.n_rows >> a.unit_log) + 2 * (int64_t)a.seqs.n_seqs;
  const int64_t items = blocks * ((int64_t)a.nq + 2 * a.nkv), most = 4 * device_sm_count();
  const unsigned ctas = (unsigned)(items < most ? items : most);
  return launch_dependent(a.k_scale ? qkv_write_kernel<HD, true> : qkv_write_kernel<HD, false>, dim3(ctas), dim3(kWrThreads), 0,
                          stream, 1u, a);
}

}  // namespace

cudaError_t launch_qkv_write(const WriteArgs &a, int32_t head_dim, cudaStream_t stream) {
  return head_dim == 256 ? launch_hd<256>(a, stream) : launch_hd<128>(a, stream);
}

}  // namespace qsa
