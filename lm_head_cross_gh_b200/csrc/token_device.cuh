// Device helpers of the token operators (token_logprobs.cu, topk_distill.cu):
// row geometry, the (reference, sum, weighted sum) state of a softmax in base 2
// and its merge, order keys of logits, a warp's selection of its k largest keys,
// and a warp's running sums over a stream of chunks.
#pragma once

#include <cstdint>

#include "ce_device.cuh"
#include "common.cuh"

namespace gh {
namespace {

constexpr float kNaN = __builtin_nanf("");
constexpr float kPosInf = __builtin_huge_valf();

// A row's bytes in 16-byte chunks, counted from its first byte rounded down to
// 16: chunks [c_lo, c_hi) lie wholly inside the row; the elements [0, h) and
// [tail, V), at most 7 (bf16) or 3 (fp32) each, do not fill one.
struct RowGeo {
  const uint8_t* src;   // first element
  const uint8_t* base;  // src rounded down to 16 bytes
  int lead;             // src - base
  int64_t c_lo, c_hi;
  int64_t h, tail;
};

template <int ES>
__device__ __forceinline__ RowGeo row_geo(const void* logits, int64_t row, int64_t ld, int64_t V) {
  RowGeo r;
  r.src = static_cast<const uint8_t*>(logits) + row * ld * ES;
  r.lead = static_cast<int>(reinterpret_cast<uintptr_t>(r.src) & 15);
  r.base = r.src - r.lead;
  const int64_t span = r.lead + V * ES;
  r.c_lo = (r.lead + 15) >> 4;
  r.c_hi = tmax<int64_t>(r.c_lo, span >> 4);
  r.h = tmin<int64_t>(V, (16 * r.c_lo - r.lead) / ES);
  r.tail = tmax<int64_t>(r.h, (16 * r.c_hi - r.lead) / ES);
  return r;
}

// The ragged-end element of a lane: lanes 0-15 the head, 16-31 the tail; -1: none.
__device__ __forceinline__ int64_t edge_element(const RowGeo& r, int64_t V, int lane) {
  if (lane < 16) return lane < r.h ? lane : -1;
  const int64_t e = r.tail + (lane - 16);
  return e < V ? e : -1;
}

// ---- softmax state -------------------------------------------------------------
// With c = log2(e) / T and y_j = x_j c - R:  s = sum 2^y_j,  t = sum 2^y_j y_j,
// and m the largest x.  R is m c rounded; y_j is one fused multiply-add, so R's
// rounding moves all terms alike.  That holds while |R| <= kFarRef (R's rounding
// is then at most 2^-5); what comes while a state has a larger R is not summed,
// and a row whose largest R is one is summed again from differences to its
// maximum (far_row).  So is a row whose largest R is less than kFarSlack above
// -kFarRef: the terms left out below that limit could count in it, while in any
// other row they are at most 2^-kFarSlack of the largest.
// R = +inf marks a NaN or +inf logit.
constexpr float kFarRef = 1048576.0f;
constexpr float kFarSlack = 256.0f;  // beyond the 2^-126 where fp32 terms end

struct SoftState {
  float m, r, s, t;
};
constexpr SoftState kNoState{-__builtin_huge_valf(), -__builtin_huge_valf(), 0.0f, 0.0f};

__device__ __forceinline__ float ref_of(float x, float c) {  // x: not NaN
  if (x == kPosInf || x == kNegInf) return x;
  return fminf(fmaxf(x * c, -3e38f), 3e38f);
}

__device__ __forceinline__ void rescale(SoftState& a, float r) {  // r >= a.r
  // a sum of 0 (its a.r may be infinite) stays 0; others have a finite distance
  const float d = a.s == 0.0f ? 0.0f : a.r - r;
  const float f = ex2(d);
  a.t = f * fmaf(a.s, d, a.t);
  a.s *= f;
  a.r = r;
}

__device__ __forceinline__ SoftState combine(SoftState a, SoftState b) {
  const float r = fmaxf(a.r, b.r);
  rescale(a, r);
  rescale(b, r);
  return {fmaxf(a.m, b.m), r, a.s + b.s, a.t + b.t};
}

// A row's distribution: log p = (x - m) / T - l, and for gradients
// p = 2^((x - sub) c - r) / s.
struct RowDist {
  float m, l;       // the largest logit; log sum exp((x - m) / T)
  float sub, r, s;
  float entropy;
  bool none;        // no distribution
};

__device__ __forceinline__ float log_p(const RowDist& d, float x, float temperature) {
  return (x - d.m) / temperature - d.l;
}

// l and the entropy from the sums about `r`.  The largest logit's own term is
// exactly 1 in sum exp((x - m) / T): it is taken out of s as it was added
// (`own`), so that l is log1p of the rest.  The rest was summed beside that term,
// so its error and l's are absolute (about 1e-7, at most 2^-20 at 50257 logits): a
// rest well below 2^-24 is not held.
__device__ __forceinline__ void finish_dist(RowDist& d, float s, float t, float y_m) {
  const float own = ex2(y_m);
  d.l = log1pf(fmaxf(s - own, 0.0f) * ex2(-y_m));
  d.entropy = d.l - kLn2 * (t / s - y_m);
}

// One of `threads` threads' part of a far row's sums of 2^y and 2^y y, y = (x - m) c:
// chains of kFarChain terms in fp32 and the chains in double.  (Terms of a row are
// alike, and one chain of n of them is off by up to n 2^-25; 31,000 by 2e-4.  One
// loop: [4096, 50257] of far rows in 484 us (bf16) and 619 (fp32), as two nested
// loops 1465 and 2351, as one fp32 chain without the double sums 470 and 490.)
constexpr int kFarChain = 32;
template <typename T, bool ENT>
__device__ __forceinline__ void far_sums(const uint8_t* src, int64_t V, float m, float c, int thread, int threads,
                                         double& s, double& t) {
  s = t = 0.0;
  float cs = 0.0f, ct = 0.0f;
  int n = 0;
#pragma unroll 8
  for (int64_t j = thread; j < V; j += threads) {
    const float y = (Elem<T>::load(src + j * Elem<T>::kBytes) - m) * c, e = ex2(y);
    cs += e;
    if (ENT && e > 0.0f) ct = fmaf(e, y, ct);
    if (++n % kFarChain == 0) {
      s += cs;
      t += ct;
      cs = ct = 0.0f;
    }
  }
  s += cs;
  t += ct;
}

// A row whose logits all lie far from 0 (lowest-value masks, tiny
// temperatures), by one warp: the maximum, then the sums of (x - max) c.
template <typename T>
__device__ __noinline__ RowDist far_row(const uint8_t* src, int64_t V, float c) {
  constexpr int ES = Elem<T>::kBytes;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  float m = kNegInf;
  for (int64_t j = lane; j < V; j += 32) m = fmaxf(m, Elem<T>::load(src + j * ES));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  double s, t;
  far_sums<T, true>(src, V, m, c, lane, 32, s, t);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  RowDist d{m, 0.0f, m, 0.0f, static_cast<float>(s), 0.0f, false};
  finish_dist(d, d.s, static_cast<float>(t), 0.0f);
  return d;
}

// The distribution from a row's merged state (the same in every lane).
template <typename T>
__device__ __forceinline__ RowDist row_dist(const SoftState& st, const uint8_t* src, int64_t V, float c) {
  if (st.r == kPosInf || st.r == kNegInf) return {0.0f, 0.0f, 0.0f, 0.0f, 1.0f, 0.0f, true};
  if (st.r > kFarRef || st.r < kFarSlack - kFarRef) return far_row<T>(src, V, c);
  RowDist d{st.m, 0.0f, 0.0f, st.r, st.s, 0.0f, false};
  finish_dist(d, st.s, st.t, fmaf(st.m, c, -st.r));
  return d;
}

// ---- order keys ------------------------------------------------------------------
// Order-preserving key of a logit that is not NaN (-0 and +0 alike); 0 is below
// every logit's key.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
// Key of (value descending, index ascending): the larger comes first.
__device__ __forceinline__ uint64_t rank_key(uint32_t key, int64_t j) {
  return (static_cast<uint64_t>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(j));
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t k = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ int64_t key_index(uint64_t key) {
  return static_cast<int64_t>(0xffffffffu - static_cast<uint32_t>(key));
}

// A warp's k largest of the keys pushed to it (k <= GH_MAX_TOP_K).  Keys at or
// below `thr` are dropped; when the buffer fills, it is cut to its k largest
// and `thr` rises to the last of them.  Keys are distinct.
constexpr int kTopBuf = 256;

struct WarpTopK {
  uint64_t* buf;  // [kTopBuf], this warp's
  uint64_t* out;  // [GH_MAX_TOP_K], this warp's
  int k, n;
  uint64_t thr;

  __device__ __forceinline__ void push(uint64_t key, bool ok) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    ok = ok && key > thr;
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    if (mask == 0) return;
    if (ok) buf[n + __popc(mask & ((1u << lane) - 1))] = key;
    n += __popc(mask);
    if (n > kTopBuf - 32) cut();
  }

  // Leaves the k largest (or all n) in out[], largest first, and in buf[].
  __device__ __forceinline__ void cut() {
    cut_keys(buf, out, n, k);
    n = tmin(n, k);
    if (n == k) thr = out[k - 1];
  }

  static __device__ __noinline__ void cut_keys(uint64_t* buf, uint64_t* out, int n, int k) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
      const uint64_t v = buf[i];
      int above = 0;
      for (int j = 0; j < n; ++j) above += buf[j] > v ? 1 : 0;
      if (above < k) out[above] = v;
    }
    __syncwarp();
    for (int i = lane; i < tmin(n, k); i += 32) buf[i] = out[i];
    __syncwarp();
  }
};

// ---- a warp's running sums ---------------------------------------------------------
// Rows stream through warps in batches of kBatch segments; a segment is one
// 16-byte load of a warp.
constexpr int kBatch = 4;
constexpr int kSegChunks = 32;  // 512 bytes
constexpr int kBatchChunks = kBatch * kSegChunks;

__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float f32_max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <typename T>
__device__ __forceinline__ uint4 max4(const uint4& a, const uint4& b);
template <>
__device__ __forceinline__ uint4 max4<uint16_t>(const uint4& a, const uint4& b) {
  return make_uint4(bf16x2_max_nan(a.x, b.x), bf16x2_max_nan(a.y, b.y), bf16x2_max_nan(a.z, b.z),
                    bf16x2_max_nan(a.w, b.w));
}
template <>
__device__ __forceinline__ uint4 max4<float>(const uint4& a, const uint4& b) {
  return make_uint4(__float_as_uint(f32_max_nan(__uint_as_float(a.x), __uint_as_float(b.x))),
                    __float_as_uint(f32_max_nan(__uint_as_float(a.y), __uint_as_float(b.y))),
                    __float_as_uint(f32_max_nan(__uint_as_float(a.z), __uint_as_float(b.z))),
                    __float_as_uint(f32_max_nan(__uint_as_float(a.w), __uint_as_float(b.w))));
}
// Largest element of a chunk; NaN if there is one.
template <typename T>
__device__ __forceinline__ float max_of4(const uint4& q);
template <>
__device__ __forceinline__ float max_of4<uint16_t>(const uint4& q) {
  const uint32_t m = bf16x2_max_nan(bf16x2_max_nan(q.x, q.y), bf16x2_max_nan(q.z, q.w));
  return f32_max_nan(bf16_lo(m), bf16_hi(m));
}
template <>
__device__ __forceinline__ float max_of4<float>(const uint4& q) {
  return f32_max_nan(f32_max_nan(__uint_as_float(q.x), __uint_as_float(q.y)),
                     f32_max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
}

// Logits below `low` add nothing to a row of |R| <= kFarRef; raised to it they
// keep y finite, so that 0 y = 0 in t.
template <typename T>
__device__ __forceinline__ uint4 clamp_low(const uint4& q, uint32_t low);
template <>
__device__ __forceinline__ uint4 clamp_low<uint16_t>(const uint4& q, uint32_t low) {
  return make_uint4(bf16x2_max(q.x, low), bf16x2_max(q.y, low), bf16x2_max(q.z, low), bf16x2_max(q.w, low));
}
template <>
__device__ __forceinline__ uint4 clamp_low<float>(const uint4& q, uint32_t low) {
  const float l = __uint_as_float(low);
  return make_uint4(__float_as_uint(fmaxf(__uint_as_float(q.x), l)), __float_as_uint(fmaxf(__uint_as_float(q.y), l)),
                    __float_as_uint(fmaxf(__uint_as_float(q.z), l)), __float_as_uint(fmaxf(__uint_as_float(q.w), l)));
}

// Largest of the warp's values; NaN if there is one.
__device__ __forceinline__ float warp_max_nan(float v) {
  float d;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
  return d;
}

// A warp's running sums: one reference for its lanes (the largest logit so
// far), so it rises seldom and the lanes' sums add without rescaling.
struct WarpSums {
  float m;         // largest logit so far (-inf: none; +inf: a NaN or +inf was seen)
  float r;         // its reference, ref_of(m)
  float2 s[2], t[2];
};

// A batch's largest logit is `m` (NaN if it has one): raise the reference.
__device__ __forceinline__ void raise(WarpSums& w, float m, float c) {
  const float top = m < kPosInf ? m : kPosInf;
  const float r = ref_of(top, c);
  const bool sums = fabsf(w.r) <= kFarRef;  // else there is nothing to rescale yet
  const float d = sums ? fmaxf(w.r - r, -2.0f * kFarRef) : 0.0f, f = ex2(d);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w.t[i] = make_float2(f * fmaf(w.s[i].x, d, w.t[i].x), f * fmaf(w.s[i].y, d, w.t[i].y));
    w.s[i] = make_float2(f * w.s[i].x, f * w.s[i].y);
  }
  w.m = top;
  w.r = r;
}

// Folds a lane's chunks of a batch into its warp's sums.  TOPK: the segments'
// largest logits go to m[].
template <typename T, bool ENT, bool TOPK>
__device__ __forceinline__ void fold_batch(WarpSums& w, const uint4 (&q)[kBatch], float c, uint32_t low,
                                           float (&m)[kBatch]) {
  constexpr int EPC = 16 / Elem<T>::kBytes;
  float bm;
  if constexpr (TOPK) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) m[i] = warp_max_nan(max_of4<T>(q[i]));
    bm = f32_max_nan(f32_max_nan(m[0], m[1]), f32_max_nan(m[2], m[3]));
  } else {
    bm = warp_max_nan(max_of4<T>(max4<T>(max4<T>(q[0], q[1]), max4<T>(q[2], q[3]))));
  }
  if (!(bm <= w.m)) raise(w, bm, c);
  if (!(fabsf(w.r) <= kFarRef)) return;
  const float2 c2 = make_float2(c, c), nr = make_float2(-w.r, -w.r);
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    float v[EPC];
    unpack16<T>(ENT ? clamp_low<T>(q[i], low) : q[i], v);
#pragma unroll
    for (int j = 0; j < EPC; j += 2) {
      const float2 y = __ffma2_rn(make_float2(v[j], v[j + 1]), c2, nr);
      const float2 e = make_float2(ex2(y.x), ex2(y.y));
      float2& a = w.s[(j / 2) & 1];
      a = __fadd2_rn(a, e);
      if constexpr (ENT) {
        float2& b = w.t[(j / 2) & 1];
        b = __ffma2_rn(e, y, b);
      }
    }
  }
}

// One more logit per lane (-inf: none) into a warp's sums: a row's ragged ends.
template <bool ENT>
__device__ __forceinline__ void fold_lanes(WarpSums& w, float x, float c) {
  const float m = warp_max_nan(x);
  if (!(m <= w.m)) raise(w, m, c);
  if (!(fabsf(w.r) <= kFarRef)) return;
  const float y = fmaxf(fmaf(x, c, -w.r), -1e30f), e = ex2(y);
  w.s[0].x += e;
  if (ENT) w.t[0].x = fmaf(e, y, w.t[0].x);
}

// Merging the warps' sums without shuffles: under a full load of global
// accesses a shuffle waits in the same queue, and a butterfly of five was
// measured at 7500 clocks.  Every lane posts its sums; one warp adds up the
// warps lane by lane, and then the 32 lanes from shared memory, in one order.
template <int W, bool ENT>
struct LaneSums {
  float top[W], ref[W];
  float s[W][32], t[ENT ? W : 1][32];
  __align__(16) float lane_s[32], lane_t[32];

  __device__ __forceinline__ void post(int warp, int lane, const WarpSums& w) {
    const float2 sa = __fadd2_rn(w.s[0], w.s[1]);
    s[warp][lane] = sa.x + sa.y;
    if (ENT) {
      const float2 ta = __fadd2_rn(w.t[0], w.t[1]);
      t[warp][lane] = ta.x + ta.y;
    }
    if (lane == 0) {
      top[warp] = w.m;
      ref[warp] = w.r;
    }
  }

  // By one warp, after a barrier; every lane gets the state.
  __device__ __forceinline__ SoftState merge(int lane) {
    SoftState v[W];
    SoftState a = kNoState;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v[i] = {top[i], ref[i], s[i][lane], ENT ? t[i][lane] : 0.0f};
      a.m = fmaxf(a.m, v[i].m);
      a.r = fmaxf(a.r, v[i].r);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      rescale(v[i], a.r);
      a.s += v[i].s;
      a.t += v[i].t;
    }
    lane_s[lane] = a.s;
    if (ENT) lane_t[lane] = a.t;
    __syncwarp();
    float4 ss = make_float4(0.0f, 0.0f, 0.0f, 0.0f), tt = ss;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 q = reinterpret_cast<const float4*>(lane_s)[i];
      ss = make_float4(ss.x + q.x, ss.y + q.y, ss.z + q.z, ss.w + q.w);
      if (ENT) {
        const float4 p = reinterpret_cast<const float4*>(lane_t)[i];
        tt = make_float4(tt.x + p.x, tt.y + p.y, tt.z + p.z, tt.w + p.w);
      }
    }
    __syncwarp();
    return {a.m, a.r, (ss.x + ss.y) + (ss.z + ss.w), (tt.x + tt.y) + (tt.z + tt.w)};
  }
};

}  // namespace
}  // namespace gh
