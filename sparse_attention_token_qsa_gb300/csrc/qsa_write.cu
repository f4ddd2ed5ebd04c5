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
// a token and a run of its heads, whose loads it issues together.  K or V in 8 bits of a
// block and a head is for as many warps as have four loads each, and up to eight: their
// maxima meet, then they write from registers (or from what they read again).  Both kinds of
// work are shared out over all CTAs alike.
//
// A chunk of 4096 rows of 16 heads over 2 x 256 into 8 bits takes 24.6 us (3.3 TB/s read and
// written, 48 % of the copy bandwidth), eight prompts of 101 to 777 rows of 32 over 8 x 128 in bf16
// 21.3 us (65 %): the launch and the chain lengths - positions - rows are 5 us of it, the rest
// waits for loads with half of the issue slots used.  Loads of a warp on their way and CTAs
// an SM holds, 4 / 3 here: 8 / 2 24.0 and 28.2 us, 4 / 4 24.7 and 21.3 (but blocks of 128
// tokens 44.8, for 38.6), 2 / 4 26.6 and 23.6, 4 / 2 26.6 and 27.4.  Single rows are a chain of
// trips to memory.
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

// Runs of heads of a token, of q and, in bf16, of K and of V; a block's K and V in 8 bits of
// every head, and log2 of the warps that take one.
struct WriteCut {
  FastDiv runs;
  int32_t q, k;
  FastDiv streams;
  int32_t warps_log;
};

constexpr int kRun = 4;  // loads of heads on their way

// A warp's (or a few warps') walk through its CTA's share of a list: every step-th item from
// the first-th on.
template <typename Count>
struct WarpWalk {
  const CachedSeqs &seqs;
  const Count &count_of;
  int64_t left, off, count;
  int32_t s, by;
  SeqView v;
  __device__ WarpWalk(const CachedSeqs &seqs_, const Count &count_of_, const FoundShare &f, int first, int by_)
      : seqs(seqs_), count_of(count_of_), left(f.share.n - first), off(f.off + first), s(f.seq), by(by_) {
    if (left <= 0) return;
    v = view_seq(seqs, s);
    count = count_of(v);
  }
  __device__ bool here() {  // to the sequence that has the item
    if (left <= 0) return false;
    while (off >= count) {
      off -= count;
      if (++s >= seqs.n_seqs) return false;
      v = view_seq(seqs, s);
      count = count_of(v);
    }
    return true;
  }
  __device__ void step() {
    left -= by;
    off += by;
  }
};

template <int HD, bool EIGHT>
__global__ void __launch_bounds__(kWrThreads, 3) qkv_write_kernel(const WriteArgs a, const WriteCut cut) {
  __shared__ ShareScratch scratch;
  __shared__ float most[kWrWarps];
  __shared__ int32_t some[kWrWarps];
  constexpr int kLanes = HD / 8, kPer = 32 / kLanes;  // lanes of a head, heads a warp takes at once
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane % kLanes, sub = lane / kLanes;
  grid_dependency_sync();

  const int ul = a.unit_log;
  // a sequence's runs, and its blocks' K and V of every head
  auto runs_of = [&](const SeqView &v) -> int64_t { return (int64_t)v.rows * cut.runs.d; };
  auto blocks_of = [&](const SeqView &v) -> int64_t {
    return v.rows == 0 ? 0 : (int64_t)(((v.ctx + v.rows - 1) >> ul) - (v.ctx >> ul) + 1) * cut.streams.d;
  };
  auto share_of = [&](auto &&count_of, bool report) {
    return find_share(a.seqs.n_seqs, kWrThreads, gridDim.x, blockIdx.x, scratch, [&](int32_t s) -> int64_t {
      if (s >= a.seqs.n_seqs) return 0;
      const SeqView v = view_seq(a.seqs, s);
      if (report && !v.ok && blockIdx.x == 0) report_error(a.status, kErrRowRange, s);
      return count_of(v);
    });
  };
  const FoundShare by_runs = share_of(runs_of, true);
  // a token's position, or -1 where its row is left alone
  auto position = [&](const SeqView &v, int32_t s, int32_t t) -> int32_t {
    const int32_t at = a.pos ? a.pos[v.row0 + (t - v.ctx)] : t;
    const bool ok = at >= 0 && at < a.table_rows;
    if (!ok) report_error(a.status, kErrRowRange, s);
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

  if constexpr (EIGHT) {
    if (a.seqs.n_seqs > 32) __syncthreads();  // the first share is read
    const FoundShare by_blocks = share_of(blocks_of, false);
    const int wl = cut.warps_log, ws = 1 << wl, group = warp >> wl, wi = warp & (ws - 1);
    for (WarpWalk<decltype(blocks_of)> walk(a.seqs, blocks_of, by_blocks, group, kWrWarps >> wl); walk.here(); walk.step()) {
      const SeqView v = walk.v;
      const int32_t nth = fast_div(cut.streams, (int32_t)walk.off), part = (int32_t)walk.off - nth * cut.streams.d;
      const bool is_k = part < a.nkv;
      const int32_t kvh = is_k ? part : part - a.nkv;
      const int32_t begin = ((v.ctx >> ul) + nth) << ul;
      const int32_t t0 = max(v.ctx, begin), t1 = (int32_t)min((int64_t)v.ctx + v.rows, (int64_t)begin + (1 << ul));
      const uint16_t *const src = (is_k ? a.k : a.v) + (int64_t)kvh * HD;
      const int64_t src_stride = is_k ? a.k_stride : a.v_stride;
      const bool norm = is_k && a.k_norm_w != nullptr;
      const HeadWeights kw(norm ? a.k_norm_w : nullptr, g);
      // kRun of the tokens from t on, ready to be held; which of them count
      uint64_t y[kRun][4];
      uint32_t good = 0u;
      auto fetch = [&](int32_t t) {
        uint4 x[kRun];
        HeadAngle turn[kRun];
        good = 0u;
#pragma unroll
        for (int b = 0; b < kRun; ++b) {
          const int32_t tb = t + (b * ws + wi) * kPer + sub;
          int32_t at = -1;
          x[b] = none;
          if (tb < t1) {
            x[b] = load_dims(src + (int64_t)(v.row0 + (tb - v.ctx)) * src_stride, g);
            at = position(v, walk.s, tb);
          }
          good |= at >= 0 ? 1u << b : 0u;
          turn[b] = angle(is_k ? at : -1);
        }
#pragma unroll
        for (int b = 0; b < kRun; ++b) {
          y[b][0] = widen(x[b].x);
          y[b][1] = widen(x[b].y);
          y[b][2] = widen(x[b].z);
          y[b][3] = widen(x[b].w);
          if (is_k) prepare_head<HD>(y[b], norm, kw.w, a.eps, turn[b]);
        }
      };
      fetch(t0);
      const int64_t slot0 = token_slot(a.seqs, walk.s, begin);  // a block lies in one page
      if (slot0 < 0) {
        if (lane == 0) report_error(a.status, kErrTokenRange, walk.s);
        continue;
      }
      float *scale = (is_k ? a.k_scale : a.v_scale) + (slot0 >> ul) * a.nkv + kvh;
      const float old = t0 > begin ? *scale : 0.f;
      uint8_t *pool = static_cast<uint8_t *>(is_k ? a.k_pool : a.v_pool) + (slot0 * a.nkv + kvh) * HD;
      const int64_t pitch = (int64_t)a.nkv * HD;
      float amax = 0.f;
      bool any = false;
      const int32_t batch = (kRun * kPer) << wl;
      for (int32_t t = t0;;) {
#pragma unroll
        for (int b = 0; b < kRun; ++b) {
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
      if (wl > 0) {
        auto meet = [&]() { asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "r"(32 << wl) : "memory"); };
        if (lane == 0) {
          most[warp] = amax;
          some[warp] = any;
        }
        meet();
        for (int w = group << wl; w < (group + 1) << wl; ++w) {
          amax = fmaxf(amax, most[w]);
          any = any || some[w];
        }
        meet();  // read before the next item's, and everyone has the old scale
      }
      if (!any) continue;
      const float now = fmaxf(old, scale_of(amax));
      if (now > old) {
        for (int32_t t = begin + wi * kPer + sub; t < t0; t += kPer << wl) {
          uint2 *at = reinterpret_cast<uint2 *>(pool + (t - begin) * pitch + 8 * g);  // (in any order)
          float z[8];
          unpack_e4m3(*at, z);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = over(z[i] * old, now);
          *at = make_uint2(pack_e4m3(z[0], z[1], z[2], z[3]), pack_e4m3(z[4], z[5], z[6], z[7]));
        }
      }
      const float inv = reciprocal(now);
      if (t0 + batch < t1) fetch(t0);  // (else the registers have them)
      for (int32_t t = t0;;) {
#pragma unroll
        for (int b = 0; b < kRun; ++b) {
          if (!((good >> b) & 1u)) continue;
          float z[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) unpair_f32(y[b][i], z[2 * i], z[2 * i + 1]);
          if (inv > 0.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] *= inv;
          } else {  // a begun block's scale that no power of two is
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = over(z[i], now);
          }
          uint8_t *at = pool + (t + (b * ws + wi) * kPer + sub - begin) * pitch;
          *reinterpret_cast<uint32_t *>(at + dim_a(g)) = pack_e4m3(z[0], z[1], z[2], z[3]);
          *reinterpret_cast<uint32_t *>(at + dim_b(g)) = pack_e4m3(z[4], z[5], z[6], z[7]);
        }
        t += batch;
        if (t >= t1) break;
        fetch(t);
      }
      __syncwarp();
      if (wi == 0 && lane == 0) *scale = now;
    }
  }

  // ---- heads streamed
  const HeadWeights qw(a.q_norm_w, g), kw(EIGHT ? nullptr : a.k_norm_w, g);
  for (WarpWalk<decltype(runs_of)> walk(a.seqs, runs_of, by_runs, warp, kWrWarps); walk.here(); walk.step()) {
    const SeqView v = walk.v;
    const int32_t j = fast_div(cut.runs, (int32_t)walk.off), run = (int32_t)walk.off - j * cut.runs.d, t = v.ctx + j;
    const int64_t row = v.row0 + j;
    // 0: q, 1: K, 2: V; the run's first head of its kind
    const int kind = EIGHT || run < cut.q ? 0 : run < cut.q + cut.k ? 1 : 2;
    const int32_t h0 = (run - (kind == 0 ? 0 : kind == 1 ? cut.q : cut.q + cut.k)) * (kRun * kPer) + sub;
    const int32_t heads = kind == 0 ? a.nq : a.nkv;
    const uint16_t *src = kind == 0 ? a.q + row * a.q_stride : kind == 1 ? a.k + row * a.k_stride : a.v + row * a.v_stride;
    src += (int64_t)h0 * HD;
    uint4 x[kRun];
#pragma unroll
    for (int b = 0; b < kRun; ++b) x[b] = h0 + b * kPer < heads ? load_dims(src + b * (kPer * HD), g) : none;
    const int32_t at = position(v, walk.s, t);
    const HeadAngle turn = angle(kind < 2 ? at : -1);
    uint16_t *dst = a.q_out + row * a.out_stride;
    if (!EIGHT && kind > 0) {
      const int64_t slot = token_slot(a.seqs, walk.s, t);
      if (slot < 0) {
        report_error(a.status, kErrTokenRange, walk.s);
        continue;
      }
      dst = static_cast<uint16_t *>(kind == 1 ? a.k_pool : a.v_pool) + slot * a.nkv * HD;
    }
    dst += (int64_t)h0 * HD;
    if (at < 0) continue;
    const bool norm = kind == 0 ? a.q_norm_w != nullptr : kind == 1 && a.k_norm_w != nullptr;
#pragma unroll
    for (int b = 0; b < kRun; ++b) {
      uint2 lo = make_uint2(x[b].x, x[b].y), hi = make_uint2(x[b].z, x[b].w);
      if (EIGHT || kind < 2) {  // (V as it is)
        uint64_t y[4] = {widen(x[b].x), widen(x[b].y), widen(x[b].z), widen(x[b].w)};
        if (EIGHT || kind == 0) prepare_head<HD>(y, norm, qw.w, a.eps, turn);
        else prepare_head<HD>(y, norm, kw.w, a.eps, turn);
        lo = make_uint2(narrow(y[0]), narrow(y[1]));
        hi = make_uint2(narrow(y[2]), narrow(y[3]));
      }
      if (h0 + b * kPer >= heads) continue;
      *reinterpret_cast<uint2 *>(dst + b * (kPer * HD) + dim_a(g)) = lo;
      *reinterpret_cast<uint2 *>(dst + b * (kPer * HD) + dim_b(g)) = hi;
    }
  }
}

template <int HD>
cudaError_t launch_hd(const WriteArgs &a, cudaStream_t stream) {
  constexpr int32_t kHeads = kRun * 256 / HD;  // of a run
  const bool eight = a.k_scale != nullptr;
  const int32_t q = (a.nq + kHeads - 1) / kHeads, k = eight ? 0 : (a.nkv + kHeads - 1) / kHeads;
  const int64_t rows = a.seqs.n_rows, n = a.seqs.n_seqs, unit = (int64_t)1 << a.unit_log;
  // the loads of a block's tokens, by the mean over the call
  const int64_t loads = ((rows / n < unit ? rows / n : unit) * HD + 255) / 256;
  const int warps_log = loads <= kRun ? 0 : loads <= 2 * kRun ? 1 : loads <= 4 * kRun ? 2 : 3;
  const WriteCut cut = {make_fast_div(q + 2 * k), q, k, make_fast_div(2 * a.nkv), warps_log};
  const int64_t items = rows * cut.runs.d + (eight ? (((rows >> a.unit_log) + 2 * n) * 2 * a.nkv) << warps_log : 0);
  const int64_t ctas = (items + kWrWarps - 1) / kWrWarps, room = 3 * device_sm_count();
  return launch_dependent(eight ? qkv_write_kernel<HD, true> : qkv_write_kernel<HD, false>, dim3((unsigned)(ctas < room ? ctas : room)),
                          dim3(kWrThreads), 0, stream, 1u, a, cut);
}

}  // namespace

cudaError_t launch_qkv_write(const WriteArgs &a, int32_t head_dim, cudaStream_t stream) {
  return head_dim == 256 ? launch_hd<256>(a, stream) : launch_hd<128>(a, stream);
}

}  // namespace qsa
