// The query and key heads of new tokens normed and rotated, K and V into the cache.
//
//   y = x / sqrt(mean(x^2) + eps) * (1 + w),  dims (i, i + 32), i < 32, turned by the
//   token's angle;  q: bf16;  K, V: bf16, or e4m3 of y / s with one scale s = 2^e for the
//   tokens of a block and a head, the least with max |y| <= 448 s.
//
// Every row is read once and written once, so HBM bounds a chunk of a prompt, if the lanes
// keep up: a head of 256 dims is 8 a lane, and its sum's shuffles, root and rotation are a
// few dozen instructions beside them.  So the first eight lanes of a head hold dims 4g to
// 4g + 3 and those 32 on, the pairs that turn together, the others 8g to 8g + 7.
//
// Query heads (and those of K and V where they are held in bf16) are streamed: a warp has
// a token and a run of its heads, whose loads it issues together.  K and V in 8 bits need a
// block's maximum first: CTAs of their own take a block's K and V of one head (four warps
// each, whose maxima meet) or, where blocks get a token or two, of four heads (a warp each).
#include "qsa_launch.h"
#include "qsa_share.cuh"
#include "qsa_tc_cache.cuh"

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

// 1 / s of a power of two in the range where both are normal numbers, else 0.
__device__ __forceinline__ float reciprocal(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x7FFFFFu) == 0u && u >= 0x00800000u && u <= 0x7E000000u ? __uint_as_float(0x7F000000u - u) : 0.f;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float rsqrt_approx(float x) {  // within 2^-22.9 of it
  float r;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two bf16 of a word, and the word of two f32.
__device__ __forceinline__ uint64_t widen(uint32_t w) { return pair_f32(lo_bf16(w), hi_bf16(w)); }
__device__ __forceinline__ uint32_t narrow(uint64_t x) {
  float lo, hi;
  unpair_f32(x, lo, hi);
  return pack_f32_bf16(lo, hi);
}

// Eight dims of a head: where lane g's two fours begin, and their bf16 words.
__device__ __forceinline__ int dim_a(int g) { return g < 8 ? 4 * g : 8 * g; }
__device__ __forceinline__ int dim_b(int g) { return g < 8 ? 4 * g + 32 : 8 * g + 4; }
__device__ __forceinline__ uint4 load_dims(const uint16_t *head, int g) {
  const uint2 a = *reinterpret_cast<const uint2 *>(head + dim_a(g)), b = *reinterpret_cast<const uint2 *>(head + dim_b(g));
  return make_uint4(a.x, a.y, b.x, b.y);
}

// A position's cosines and sines of the dims that a lane turns.
struct HeadAngle {
  uint2 cos, sin;
  bool on;
};

// A head's weights in f32, 1 added.
struct HeadWeights {
  uint64_t w[4];
  __device__ HeadWeights(const uint16_t *p, int g) {
    const uint4 x = p ? load_dims(p, g) : make_uint4(0, 0, 0, 0);
    const uint64_t one = pair_f32(1.f, 1.f);
    w[0] = add2(widen(x.x), one);
    w[1] = add2(widen(x.y), one);
    w[2] = add2(widen(x.z), one);
    w[3] = add2(widen(x.w), one);
  }
};

// The head of one token, normed and turned by its angle.  Every lane of the warp.
template <int HD>
__device__ __forceinline__ void prepare_head(uint64_t (&x)[4], bool norm, const uint64_t (&w)[4], float eps, const HeadAngle &turn) {
  float lo, hi;
  unpair_f32(fma2(x[3], x[3], fma2(x[2], x[2], fma2(x[1], x[1], mul2(x[0], x[0])))), lo, hi);
  float sum = lo + hi;
#pragma unroll
  for (int o = HD / 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (norm) {
    const float r = rsqrt_approx(fmaf(sum, 1.f / HD, eps));
    const uint64_t r2 = pair_f32(r, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul2(mul2(x[i], r2), w[i]);
  }
  if (turn.on) {
    const uint64_t minus = pair_f32(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t c = widen(i ? turn.cos.y : turn.cos.x), s = widen(i ? turn.sin.y : turn.sin.x);
      const uint64_t a = x[i], b = x[i + 2];
      x[i] = fma2(a, c, mul2(mul2(b, s), minus));
      x[i + 2] = fma2(b, c, mul2(a, s));
    }
  }
}

// How a launch shares its work out.
struct WriteCut {
  int32_t kv_ctas;   // CTAs that take K and V in 8 bits, before those that stream
  int32_t kv_parts;  // items of a block there
  int32_t few;       // a warp takes K or V of a head alone, not four
  FastDiv runs;      // runs of heads of a token
};

constexpr int kRun = 8;  // loads of a run of heads

template <int HD, bool EIGHT>
__global__ void __launch_bounds__(kWrThreads, EIGHT ? 2 : 3) qkv_write_kernel(const WriteArgs a, const WriteCut cut) {
  __shared__ ShareScratch scratch;
  __shared__ float most[kWrWarps];
  __shared__ int32_t some[kWrWarps];
  constexpr int kLanes = HD / 8, kPer = 32 / kLanes;  // lanes of a head, heads a warp takes at once
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane % kLanes, sub = lane / kLanes;
  grid_dependency_sync();

  const int ul = a.unit_log;
  const bool kv = EIGHT && (int32_t)blockIdx.x < cut.kv_ctas;
  // what a sequence has in the list of this CTA's kind: blocks' items, or tokens' runs
  auto count_of = [&](const SeqView &v) -> int64_t {
    if (v.rows == 0) return 0;
    return kv ? (int64_t)(((v.ctx + v.rows - 1) >> ul) - (v.ctx >> ul) + 1) * cut.kv_parts : (int64_t)v.rows * cut.runs.d;
  };
  FoundShare f = find_share(a.seqs.n_seqs, kWrThreads, kv ? cut.kv_ctas : gridDim.x - cut.kv_ctas,
                            kv ? blockIdx.x : blockIdx.x - cut.kv_ctas, scratch, [&](int32_t s) -> int64_t {
                              if (s >= a.seqs.n_seqs) return 0;
                              const SeqView v = view_seq(a.seqs, s);
                              if (!v.ok && blockIdx.x == 0) report_error(a.status, kErrRowRange, s);
                              return count_of(v);
                            });
  SeqView v = {0, 0, 0, false};
  int64_t count = 0;
  if (f.share.n > 0) {
    v = view_seq(a.seqs, f.seq);
    count = count_of(v);
  }
  auto walk = [&](int64_t &off) -> bool {  // to the sequence that has item `off`
    while (off >= count) {
      off -= count;
      if (++f.seq >= a.seqs.n_seqs) return false;
      v = view_seq(a.seqs, f.seq);
      count = count_of(v);
    }
    return true;
  };
  // a token's position, or -1 where its row is left alone
  auto position = [&](int32_t t) -> int32_t {
    const int32_t at = a.pos ? a.pos[v.row0 + (t - v.ctx)] : t;
    const bool ok = at >= 0 && at < a.table_rows;
    if (!ok) report_error(a.status, kErrRowRange, f.seq);
    return ok ? at : -1;
  };
  auto angle = [&](int32_t at) -> HeadAngle {
    HeadAngle h = {make_uint2(0, 0), make_uint2(0, 0), at >= 0 && g < 8};
    if (h.on) {
      h.cos = *reinterpret_cast<const uint2 *>(a.cos_t + (int64_t)at * kRot + 4 * g);
      h.sin = *reinterpret_cast<const uint2 *>(a.sin_t + (int64_t)at * kRot + 4 * g);
    }
    return h;
  };
  const uint4 none = make_uint4(0, 0, 0, 0);

  const HeadWeights kw(a.k_norm_w, g);
  if (!kv) {
    // ---- heads streamed
    const int32_t heads = a.nq + (EIGHT ? 0 : 2 * a.nkv);
    const HeadWeights qw(a.q_norm_w, g);
    int64_t off = f.off + warp;
    for (int64_t left = f.share.n - warp; left > 0; left -= kWrWarps, off += kWrWarps) {
      if (!walk(off)) return;
      const int32_t j = fast_div(cut.runs, (int32_t)off), first = ((int32_t)off - j * cut.runs.d) * (kRun * kPer), h0 = first + sub;
      const int32_t t = v.ctx + j;
      const int64_t row = v.row0 + j;
      uint4 x[kRun];
#pragma unroll
      for (int b = 0; b < kRun; ++b) {
        const int32_t h = h0 + b * kPer;
        const uint16_t *src = a.q + row * a.q_stride + (int64_t)h * HD;
        if (!EIGHT && h >= a.nq)
          src = h < a.nq + a.nkv ? a.k + row * a.k_stride + (int64_t)(h - a.nq) * HD
                                 : a.v + row * a.v_stride + (int64_t)(h - a.nq - a.nkv) * HD;
        x[b] = h < heads ? load_dims(src, g) : none;
      }
      const int32_t at = position(t);
      const HeadAngle turn = angle(at);
      int64_t slot = -1;
      if (!EIGHT && first + kRun * kPer > a.nq) {
        slot = token_slot(a.seqs, f.seq, t);
        if (slot < 0) report_error(a.status, kErrTokenRange, f.seq);
      }
#pragma unroll
      for (int b = 0; b < kRun; ++b) {
        const int32_t h = h0 + b * kPer;
        if (first + b * kPer >= heads) break;
        const bool is_q = EIGHT || h < a.nq, is_v = !EIGHT && h >= a.nq + a.nkv;
        uint64_t y[4] = {widen(x[b].x), widen(x[b].y), widen(x[b].z), widen(x[b].w)};
        HeadAngle mine = turn;
        bool norm = a.q_norm_w != nullptr;
        if constexpr (!EIGHT) {
          if (!is_q) norm = a.k_norm_w != nullptr && !is_v;
          mine.on = turn.on && !is_v;
          uint64_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = is_q ? qw.w[i] : kw.w[i];
          prepare_head<HD>(y, norm, w, a.eps, mine);
        } else {
          prepare_head<HD>(y, norm, qw.w, a.eps, mine);
        }
        if (h >= heads || at < 0) continue;
        uint2 lo = make_uint2(x[b].x, x[b].y), hi = make_uint2(x[b].z, x[b].w);  // V as it is
        if (!is_v) {
          lo = make_uint2(narrow(y[0]), narrow(y[1]));
          hi = make_uint2(narrow(y[2]), narrow(y[3]));
        }
        uint16_t *dst = a.q_out + row * a.out_stride + (int64_t)h * HD;
        if (!is_q) {
          if (slot < 0) continue;
          dst = static_cast<uint16_t *>(is_v ? a.v_pool : a.k_pool) + (slot * a.nkv + (h - a.nq - (is_v ? a.nkv : 0))) * HD;
        }
        *reinterpret_cast<uint2 *>(dst + dim_a(g)) = lo;
        *reinterpret_cast<uint2 *>(dst + dim_b(g)) = hi;
      }
    }
    return;
  }
  if constexpr (EIGHT) {
    // ---- K (warps 0 to 3) and V (4 to 7) of a block and a head: its scale, then its values
    constexpr int kHeld = 4;  // loads of heads on their way
    const bool is_k = warp < 4;
    const int wi = cut.few ? 0 : warp & 3, ws = cut.few ? 1 : 4;  // this warp's place among those of its head
    int64_t off = f.off;
    for (int64_t left = f.share.n; left > 0; --left, ++off) {
      if (!walk(off)) return;
      const int32_t nth = (int32_t)(off / cut.kv_parts), part = (int32_t)(off - (int64_t)nth * cut.kv_parts);
      const int32_t kvh = cut.few ? 4 * part + (warp & 3) : part;
      if (kvh >= a.nkv) continue;  // (a warp alone: no barrier below)
      const int32_t begin = ((v.ctx >> ul) + nth) << ul;
      const int32_t t0 = max(v.ctx, begin), t1 = (int32_t)min((int64_t)v.ctx + v.rows, (int64_t)begin + (1 << ul));
      const int32_t step = ws * kPer;
      // kHeld of this warp's tokens from t on, ready to be held; which of them count
      uint64_t y[kHeld][4];
      uint32_t good = 0u;
      auto fetch = [&](int32_t t) {
        uint4 x[kHeld];
        int32_t at[kHeld];
        good = 0u;
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
          const int32_t tb = t + b * step + sub;
          const int64_t row = v.row0 + (tb - v.ctx);
          at[b] = -1;
          x[b] = none;
          if (tb < t1) {
            x[b] = load_dims((is_k ? a.k + row * a.k_stride : a.v + row * a.v_stride) + (int64_t)kvh * HD, g);
            at[b] = position(tb);
          }
          good |= at[b] >= 0 ? 1u << b : 0u;
        }
        HeadAngle turn[kHeld];
        if (is_k) {
#pragma unroll
          for (int b = 0; b < kHeld; ++b) turn[b] = angle(at[b]);
        }
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
          y[b][0] = widen(x[b].x);
          y[b][1] = widen(x[b].y);
          y[b][2] = widen(x[b].z);
          y[b][3] = widen(x[b].w);
          if (is_k) prepare_head<HD>(y[b], a.k_norm_w != nullptr, kw.w, a.eps, turn[b]);
        }
      };
      const int32_t first = t0 + wi * kPer, batch = kHeld * step;
      const bool once = first + batch >= t1;  // what this warp has fits its registers
      fetch(first);
      const int64_t slot0 = token_slot(a.seqs, f.seq, begin);  // a block lies in one page
      if (slot0 < 0) {
        if (lane == 0) report_error(a.status, kErrTokenRange, f.seq);
        continue;
      }
      float *scale = (is_k ? a.k_scale : a.v_scale) + (slot0 >> ul) * a.nkv + kvh;
      const float old = t0 > begin ? *scale : 0.f;
      uint8_t *pool = static_cast<uint8_t *>(is_k ? a.k_pool : a.v_pool) + (slot0 * a.nkv + kvh) * HD;
      const int64_t pitch = (int64_t)a.nkv * HD;
      float amax = 0.f;
      bool any = false;
      for (int32_t t = first;;) {
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
          if (!((good >> b) & 1u)) continue;
          any = true;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float lo, hi;
            unpair_f32(y[b][i], lo, hi);
            lo = fabsf(lo);
            hi = fabsf(hi);
            amax = fmaxf(amax, fmaxf(lo < INFINITY ? lo : 0.f, hi < INFINITY ? hi : 0.f));
          }
        }
        t += batch;
        if (t >= t1) break;
        fetch(t);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      any = __any_sync(0xffffffffu, any);
      if (!cut.few) {
        auto meet = [&]() { asm volatile("barrier.cta.sync %0, 128;" ::"r"(is_k ? 1 : 2) : "memory"); };
        if (lane == 0) {
          most[warp] = amax;
          some[warp] = any;
        }
        meet();
        const int w0 = warp & 4;
        amax = fmaxf(fmaxf(most[w0], most[w0 + 1]), fmaxf(most[w0 + 2], most[w0 + 3]));
        any = some[w0] || some[w0 + 1] || some[w0 + 2] || some[w0 + 3];
        meet();  // read before the next item's, and everyone has the old scale
      }
      if (!any) continue;
      const float now = fmaxf(old, scale_of(amax));
      if (now > old) {
        for (int32_t t = begin + wi * kPer + sub; t < t0; t += step) {
          uint2 *at = reinterpret_cast<uint2 *>(pool + (t - begin) * pitch + 8 * g);  // (in any order)
          float z[8];
          unpack_e4m3(*at, z);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = over(z[i] * old, now);
          *at = make_uint2(pack_e4m3(z[0], z[1], z[2], z[3]), pack_e4m3(z[4], z[5], z[6], z[7]));
        }
      }
      const float inv = reciprocal(now);
      if (!once) fetch(first);
      for (int32_t t = first;;) {
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
          if (!((good >> b) & 1u)) continue;
          float z[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) unpair_f32(y[b][i], z[2 * i], z[2 * i + 1]);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = inv > 0.f ? z[i] * inv : over(z[i], now);
          uint8_t *at = pool + (t + b * step + sub - begin) * pitch;
          *reinterpret_cast<uint32_t *>(at + dim_a(g)) = pack_e4m3(z[0], z[1], z[2], z[3]);
          *reinterpret_cast<uint32_t *>(at + dim_b(g)) = pack_e4m3(z[4], z[5], z[6], z[7]);
        }
        t += batch;
        if (t >= t1) break;
        fetch(t);
      }
      if (wi == 0 && lane == 0) *scale = now;
    }
  }
}

template <int HD>
cudaError_t launch_hd(const WriteArgs &a, cudaStream_t stream) {
  constexpr int kPer = 256 / HD;
  const bool eight = a.k_scale != nullptr;
  const int64_t rows = a.seqs.n_rows, n = a.seqs.n_seqs;
  const int32_t heads = a.nq + (eight ? 0 : 2 * a.nkv);
  WriteCut cut = {0, 0, 0, make_fast_div((heads + kRun * kPer - 1) / (kRun * kPer))};
  const int64_t room = (eight ? 2 : 3) * device_sm_count();
  int64_t streams = (rows * cut.runs.d + kWrWarps - 1) / kWrWarps;  // CTAs with a run a warp
  if (eight) {
    cut.few = rows <= 4 * n;  // tokens a block gets, by the mean over the call
    cut.kv_parts = cut.few ? (a.nkv + 3) / 4 : a.nkv;
    const int64_t items = ((rows >> a.unit_log) + 2 * n) * cut.kv_parts;
    // by the bytes that are read and written, 3 a value of K and V, 4 one of q, and as much
    // again of K and V for their waits
    const int64_t part = room * 12 * a.nkv / (12 * a.nkv + 4 * a.nq) + 1;
    cut.kv_ctas = (int32_t)(items < part ? items : part);
  }
  if (streams > room - cut.kv_ctas) streams = room - cut.kv_ctas;
  return launch_dependent(eight ? qkv_write_kernel<HD, true> : qkv_write_kernel<HD, false>, dim3((unsigned)(cut.kv_ctas + streams)),
                          dim3(kWrThreads), 0, stream, 1u, a, cut);
}

}  // namespace

cudaError_t launch_qkv_write(const WriteArgs &a, int32_t head_dim, cudaStream_t stream) {
  return head_dim == 256 ? launch_hd<256>(a, stream) : launch_hd<128>(a, stream);
}

}  // namespace qsa
