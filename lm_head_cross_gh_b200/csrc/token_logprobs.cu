// Log-probabilities of given tokens with the row's entropy, log-sum-exp and
// most probable alternatives, and their gradient.
//
// For a row x of V logits, temperature T and c = log2(e) / T, with a reference
// R near its largest x c,
//     y_j = x_j c - R,   s = sum_j 2^y_j,   t = sum_j 2^y_j y_j,
//     log p_j = ln 2 (y_j - log2 s),   lse = ln 2 (R + log2 s),
//     entropy = ln 2 (log2 s - t / s)
// (a term with 2^y = 0 adds nothing to t, so -inf logits are 0 log 0 = 0).
// The alternatives are the top_k logits by (value descending, index
// ascending); the temperature does not change their order.
//
// The forward (logprobs_ring_kernel) reads every logit once.  A row is cut
// into segments of 128 bytes; the thread that sums a segment also has its
// largest logit, whose key it keeps in shared memory.  The k largest logits lie
// in the k segments that come first by (largest logit descending, position
// ascending): any other segment's logits have k segment maxima before them.
// So the alternatives cost one key per segment during the pass, a selection
// among V / 64 (bf16) keys by one warp, and k segments read again from L2.
#include <algorithm>
#include <cstring>

#include "linear_ce.h"
#include "profile.h"
#include "token_device.cuh"
#include "token_ops.h"

namespace gh {

namespace {

// ---------------------------------------------------------------------------
// Forward: one persistent CTA per SM streams units (a row, or a slice of one)
// through a ring of 16 KiB pieces, as the cross-entropy ring does:
//   warp 16      producer: bulk copies into the next free slot
//   warps 0-15   consumers, four groups of four warps; piece n goes to group
//                n % 4, a thread takes one segment (8 chunks) into registers,
//                frees the slot and folds the segment into its state
//   warps 17-20  finalizers, unit k to warp 17 + k % 4: merge the 512 thread
//                states with the ragged ends, pick the alternatives, write
// ---------------------------------------------------------------------------

constexpr int kLpWarps = 16;
constexpr int kLpGroups = 4;
constexpr int kLpGroupWarps = kLpWarps / kLpGroups;
constexpr int kLpGroupThreads = 32 * kLpGroupWarps;
constexpr int kLpFinalizers = 4;
constexpr int kLpThreads = 32 * (kLpWarps + 1 + kLpFinalizers);
constexpr int kLpPieceBytes = 16384;
constexpr int kLpPieceChunks = kLpPieceBytes / 16;
constexpr int kSegChunks = 8;  // 128 bytes
constexpr int kPieceSegs = kLpPieceChunks / kSegChunks;
static_assert(kPieceSegs == kLpGroupThreads, "one segment per thread of a group");
// Ring slots: with alternatives part of shared memory holds the segments' keys.
template <bool TOPK>
constexpr int kLpSlots = TOPK ? 8 : 12;
constexpr int kLpMaxSegs = 3584;  // segments of a unit whose keys fit beside 8 slots

struct LpShared {
  uint64_t full[12], empty[12];
  uint64_t rowfull[kLpFinalizers], rowempty[kLpFinalizers];
  float2 part_rs[kLpFinalizers][kLpWarps][32];
  float part_t[kLpFinalizers][kLpWarps][32];
  int abort;
};
struct LpTopShared {
  uint64_t buf[kLpFinalizers][kTopBuf];
  uint64_t out[kLpFinalizers][GH_MAX_TOP_K];
  int list[kLpFinalizers][GH_MAX_TOP_K];
};
constexpr int kLpHdrBytes = (static_cast<int>(sizeof(LpShared)) + 127) / 128 * 128;
constexpr int kLpTopBytes = (static_cast<int>(sizeof(LpTopShared)) + 127) / 128 * 128;

template <bool TOPK>
constexpr int lp_smem_bytes(int segs) {
  return kLpHdrBytes + kLpSlots<TOPK> * kLpPieceBytes + (TOPK ? kLpTopBytes + kLpFinalizers * 4 * segs : 0);
}
static_assert(lp_smem_bytes<true>(kLpMaxSegs) <= 227 * 1024 && lp_smem_bytes<false>(0) <= 227 * 1024, "");

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

// Folds a segment (N chunks in registers) into a thread's state; returns its
// largest logit.
template <typename T, bool ENT, int N>
__device__ __forceinline__ float fold_segment(SoftState& st, const uint4 (&q)[N], float c, uint32_t low) {
  constexpr int EPC = 16 / Elem<T>::kBytes;
  uint4 m4 = q[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m4 = max4<T>(m4, q[i]);
  const float cm = max_of4<T>(m4);
  if (!(cm < kPosInf)) {
    st = {kPosInf, 0.0f, 0.0f};
    return cm;
  }
  const float r = ref_of(cm, c);
  if (r > st.r) rescale(st, r);
  if (!(r >= -kFarRef && st.r <= kFarRef)) return cm;
  const float2 c2 = make_float2(c, c), nr = make_float2(-st.r, -st.r);
  float2 s[4], t[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 2; ++i) t[i] = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float v[EPC];
    unpack16<T>(ENT ? clamp_low<T>(q[i], low) : q[i], v);
#pragma unroll
    for (int j = 0; j < EPC; j += 2) {
      const float2 y = __ffma2_rn(make_float2(v[j], v[j + 1]), c2, nr);
      const float2 e = make_float2(ex2(y.x), ex2(y.y));
      float2& a = s[(i * EPC / 2 + j / 2) & 3];
      a = __fadd2_rn(a, e);
      if constexpr (ENT) {
        float2& b = t[(j / 2) & 1];
        b = __ffma2_rn(e, y, b);
      }
    }
  }
  const float2 sa = __fadd2_rn(__fadd2_rn(s[0], s[1]), __fadd2_rn(s[2], s[3]));
  st.s += sa.x + sa.y;
  if constexpr (ENT) {
    const float2 tb = __fadd2_rn(t[0], t[1]);
    st.t += tb.x + tb.y;
  }
  return cm;
}

// Where unit u lies: row, slice, and its chunks of the row.
struct Unit {
  int64_t row;
  int slice;
  int64_t c0, c1;  // chunks [c0, c1) of the row
};

__device__ __forceinline__ int64_t unit_row(const StatArgs& a, int64_t u) { return a.slices == 1 ? u : u / a.slices; }

__device__ __forceinline__ Unit unit_of(const StatArgs& a, int64_t u, int64_t row, const RowGeo& r) {
  Unit w;
  w.row = row;
  w.slice = static_cast<int>(u - row * a.slices);
  const int64_t per = static_cast<int64_t>(a.slice_segs) * kSegChunks;
  w.c0 = tmin(r.c_hi, r.c_lo + w.slice * per);
  w.c1 = w.slice == a.slices - 1 ? r.c_hi : tmin(r.c_hi, w.c0 + per);
  return w;
}

// A unit's chunk count alone (what the consumers need of it).
template <int ES>
__device__ __forceinline__ int unit_chunks(const StatArgs& a, int64_t u) {
  const int64_t row = unit_row(a, u);
  const uint32_t lead = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a.logits) + static_cast<uintptr_t>(row * a.ld) * ES) & 15u;
  const int lo = static_cast<int>((lead + 15) >> 4);
  const int n = tmax(0, static_cast<int>((lead + a.V * ES) >> 4) - lo);
  if (a.slices == 1) return n;
  const int slice = static_cast<int>(u - row * a.slices), per = a.slice_segs * kSegChunks;
  const int64_t from = static_cast<int64_t>(slice) * per;
  const int left = static_cast<int>(tmax<int64_t>(0, n - from));
  return slice == a.slices - 1 ? left : tmin(left, per);
}

// Rows that count: 1; ignored: 0; an index outside [0, V): -1.
__device__ __forceinline__ int row_kind(const StatArgs& a, int64_t row) {
  if (a.flags) return a.flags[row];
  const int64_t t = a.lp.index[row];
  if (t == a.lp.ignore_index) return 0;
  return t >= 0 && t < a.V ? 1 : -1;
}

// Outputs of a row that does not count (by one warp).
__device__ __forceinline__ void write_no_row(const LogprobArgs& o, int64_t row, int kind) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const float v = kind < 0 ? kNaN : 0.0f;
  if (lane == 0) {
    o.logprob[row] = o.entropy[row] = o.lse[row] = v;
    if (kind < 0) record_status(GH_ERR_TARGET_RANGE);
  }
  for (int k = lane; k < o.top_k; k += 32) {
    o.top_logprob[row * o.top_k + k] = kind < 0 ? kNaN : kNegInf;
    o.top_index[row * o.top_k + k] = -1;
  }
}

// Outputs of a row that counts, from its distribution and its alternatives'
// keys, largest first (by one warp).
template <typename T>
__device__ __forceinline__ void write_row(const LogprobArgs& o, int64_t row, const RowDist& d, float xt,
                                          const uint64_t* top) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  if (lane == 0) {
    o.logprob[row] = d.none ? kNaN : kLn2 * log2_p<T>(d, xt, o.c);
    o.entropy[row] = d.none ? kNaN : kLn2 * (d.l2s - d.ts);
    o.lse[row] = d.none ? kNaN : dist_lse(d, o.temperature);
  }
  for (int k = lane; k < o.top_k; k += 32) {
    o.top_logprob[row * o.top_k + k] = d.none ? kNaN : kLn2 * log2_p<T>(d, key_value(top[k]), o.c);
    o.top_index[row * o.top_k + k] = d.none ? -1 : key_index(top[k]);
  }
}

// The first k segments by (key descending, position ascending) of `segs` keys
// (padded with zeros to a multiple of 128): their positions into list[],
// returns how many and, in thr, a key that k of all the logits reach (0 where
// fewer segments than k exist).  The k-th largest key is found bit by bit,
// stopping as soon as a prefix has exactly k keys at or above it; bf16 keys
// differ in their upper 16 bits only.
template <typename T>
__device__ __forceinline__ int pick_segments(const uint32_t* keys, int segs, int k, int* list, uint32_t* thr) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  if (segs <= k) {
    for (int i = lane; i < segs; i += 32) list[i] = i;
    *thr = 0;
    __syncwarp();
    return segs;
  }
  const uint4* k4 = reinterpret_cast<const uint4*>(keys);
  const int n4 = (segs + 127) / 128 * 32;
  uint32_t key = 0;
  constexpr int kLastBit = Elem<T>::kBytes == 2 ? 16 : 0;
  for (int bit = 31; bit >= kLastBit; --bit) {
    const uint32_t cand = key | (1u << bit);
    int n = 0;
    for (int i = lane; i < n4; i += 32) {
      const uint4 v = k4[i];
      n += (v.x >= cand) + (v.y >= cand) + (v.z >= cand) + (v.w >= cand);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= k) key = cand;
    if (n == k) break;
  }
  // For bf16 a negative value's key ends in ones; compare on the kept bits.
  const uint32_t mask = kLastBit ? 0xffff0000u : 0xffffffffu;
  int above = 0;
  for (int i = lane; i < n4; i += 32) {
    const uint4 v = k4[i];
    above += ((v.x & mask) > key) + ((v.y & mask) > key) + ((v.z & mask) > key) + ((v.w & mask) > key);
  }
  int left = k - __reduce_add_sync(0xffffffffu, above);  // how many of the equal ones, in order
  int n = 0;
  const uint32_t below = (1u << lane) - 1;
  for (int i = 0; i < segs && n < k; i += 32) {
    const uint32_t v = i + lane < segs ? keys[i + lane] & mask : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, v == key && i + lane < segs);
    const bool take = v > key || (v == key && i + lane < segs && __popc(eq & below) < left);
    const uint32_t got = __ballot_sync(0xffffffffu, take);
    if (take) list[n + __popc(got & below)] = i + lane;
    n += __popc(got);
    left -= tmin(left, __popc(eq));
  }
  *thr = key;
  __syncwarp();
  return n;
}

// Pushes the logits of the listed segments of a unit (chunks from c0 on).
template <typename T>
__device__ __forceinline__ void push_segments(WarpTopK& top, const RowGeo& r, const Unit& w, const int* list, int n) {
  constexpr int ES = Elem<T>::kBytes, EPC = 16 / ES;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  auto chunk_of = [&](int i) -> int64_t {
    const int j = i + (lane >> 3);
    return j < n ? w.c0 + static_cast<int64_t>(list[j]) * kSegChunks + (lane & 7) : w.c1;
  };
  auto load = [&](int64_t c) {
    return c < w.c1 ? __ldcg(reinterpret_cast<const uint4*>(r.base + 16 * c)) : make_uint4(0, 0, 0, 0);
  };
  int64_t c = chunk_of(0);
  uint4 q = load(c);
  for (int i = 0; i < n; i += 4) {
    const int64_t cn = chunk_of(i + 4);
    const uint4 qn = load(cn);
    float v[EPC];
    unpack16<T>(q, v);
    const int64_t j0 = (16 * c - r.lead) / ES;
#pragma unroll
    for (int e = 0; e < EPC; ++e) top.push(rank_key(order_key(v[e]), j0 + e), c < w.c1);
    c = cn;
    q = qn;
  }
}

template <typename T, bool ENT, bool TOPK>
__global__ void __launch_bounds__(kLpThreads, 1) logprobs_ring_kernel(StatArgs a) {
  constexpr int ES = Elem<T>::kBytes;
  constexpr uint32_t kSlots = kLpSlots<TOPK>;
  extern __shared__ __align__(128) uint8_t smem[];
  LpShared& sh = *reinterpret_cast<LpShared*>(smem);
  uint8_t* ring = smem + kLpHdrBytes;
  LpTopShared& tsh = *reinterpret_cast<LpTopShared*>(ring + kSlots * kLpPieceBytes);
  uint32_t* seg_keys = reinterpret_cast<uint32_t*>(ring + kSlots * kLpPieceBytes + kLpTopBytes);
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t G = gridDim.x, first = blockIdx.x, units = a.B * a.slices;

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kLpGroupWarps);
    }
    for (int i = 0; i < kLpFinalizers; ++i) {
      mbar_init(&sh.rowfull[i], kLpWarps);
      mbar_init(&sh.rowempty[i], 1);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  __syncthreads();

  volatile int* abort_flag = &sh.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (*abort_flag) return false;
    if (mbar_wait(bar, parity)) return true;
    *abort_flag = 1;
    return false;
  };
  auto kind_of = [&](int64_t u) -> int { return u < units ? row_kind(a, unit_row(a, u)) : 0; };

  if (warp == kLpWarps) {
    // ---------------- producer ----------------
    if (lane == 0) {
      uint32_t n = 0;  // pieces issued
      int kind = kind_of(first);
      for (int64_t u = first; u < units; u += G) {
        const int next = kind_of(u + G);
        if (kind > 0) {
          const int64_t row = unit_row(a, u);
          const RowGeo r = row_geo<ES>(a.logits, row, a.ld, a.V);
          const Unit w = unit_of(a, u, row, r);
          for (int64_t c0 = w.c0; c0 < w.c1; c0 += kLpPieceChunks, ++n) {
            const uint32_t s = n % kSlots;
            if (!wait(&sh.empty[s], ((n / kSlots) & 1) ^ 1)) break;
            const uint32_t bytes = 16u * static_cast<uint32_t>(tmin<int64_t>(kLpPieceChunks, w.c1 - c0));
            mbar_arrive_expect_tx(&sh.full[s], bytes);
            bulk_g2s(ring + s * kLpPieceBytes, r.base + 16 * c0, bytes, &sh.full[s]);
          }
        }
        if (*abort_flag) break;
        kind = next;
      }
      if (*abort_flag) {  // the copies still in flight land before the CTA exits
        for (uint32_t k = (n > kSlots ? n - kSlots : 0); k < n; ++k)
          (void)mbar_wait(&sh.full[k % kSlots], (k / kSlots) & 1);
      }
    }
    return;
  }

  if (warp > kLpWarps) {
    // ---------------- finalizers ----------------
    const uint32_t f = warp - kLpWarps - 1;
    uint32_t k = 0, i = 0;  // units that count, units
    int kind = kind_of(first);
    for (int64_t u = first; u < units; u += G, ++i) {
      const int next = kind_of(u + G);
      if (kind <= 0) {
        if (!a.part && i % kLpFinalizers == f) write_no_row(a.lp, unit_row(a, u), kind);
        kind = next;
        continue;
      }
      kind = next;
      if (k % kLpFinalizers != f) {
        ++k;
        continue;
      }
      const int64_t row = unit_row(a, u);
      const RowGeo r = row_geo<ES>(a.logits, row, a.ld, a.V);
      const Unit w = unit_of(a, u, row, r);
      int64_t e = edge_element(r, a.V, lane);
      if (lane < 16 ? w.slice != 0 : w.slice != a.slices - 1) e = -1;
      const float edge = e >= 0 ? Elem<T>::load(r.src + e * ES) : kNegInf;
      float xt = 0.0f;
      if (!a.part) xt = Elem<T>::load(r.src + a.lp.index[row] * ES);
      const bool ok = __all_sync(0xffffffffu, wait(&sh.rowfull[f], (k / kLpFinalizers) & 1));
      ++k;
      if (!ok) break;
      // this lane's 16 thread states, largest reference first
      SoftState st = state_of_element(edge, a.c);
      float m = st.r;
      float2 rs[kLpWarps];
#pragma unroll
      for (int v = 0; v < kLpWarps; ++v) {
        rs[v] = sh.part_rs[f][v][lane];
        m = fmaxf(m, rs[v].x);
      }
      rescale(st, m);
#pragma unroll
      for (int v = 0; v < kLpWarps; ++v) {
        SoftState o{rs[v].x, rs[v].y, ENT ? sh.part_t[f][v][lane] : 0.0f};
        rescale(o, m);
        st.s += o.s;
        st.t += o.t;
      }
      st = warp_combine(st);
      WarpTopK top{};
      if constexpr (TOPK) {
        uint32_t* keys = seg_keys + f * a.seg_cap;
        const int segs = static_cast<int>((w.c1 - w.c0 + kSegChunks - 1) / kSegChunks);
        for (int j = segs + lane; j < (segs + 127) / 128 * 128; j += 32) keys[j] = 0;
        __syncwarp();
        uint32_t thr;
        const int n = pick_segments<T>(keys, segs, a.top_k, tsh.list[f], &thr);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.rowempty[f]);
        top.buf = tsh.buf[f];
        top.out = tsh.out[f];
        top.k = a.top_k;
        top.n = 0;
        top.thr = thr ? (static_cast<uint64_t>(thr) << 32) - 1 : 0;
        push_segments<T>(top, r, w, tsh.list[f], n);
        top.push(rank_key(order_key(edge), e), e >= 0);
        top.cut();
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.rowempty[f]);
      }
      if (a.part) {
        if (lane == 0) a.part[u] = make_float4(st.r, st.s, st.t, 0.0f);
        if constexpr (TOPK)
          for (int j = lane; j < a.top_k; j += 32) a.part_keys[u * a.top_k + j] = j < top.n ? top.out[j] : 0;
      } else {
        write_row<T>(a.lp, row, row_dist<T>(st, r.src, a.V, a.c), xt, TOPK ? top.out : nullptr);
      }
      __syncwarp();
    }
    return;
  }

  // ---------------- consumers ----------------
  const int grp = warp / kLpGroupWarps;
  const int gtid = static_cast<int>(threadIdx.x) - grp * kLpGroupThreads;
  constexpr uint32_t kGroupSlots = kSlots / kLpGroups;  // a group's slots: grp, grp + 4, ...
  static_assert(kSlots % kLpGroups == 0, "a slot always serves the same group");
  uint32_t turn = static_cast<uint32_t>(grp);  // pieces of this unit before the group's next one
  uint32_t gs = 0, gphase = 0;                 // the group's next slot and its phase
  uint32_t j = 0, jphase = 1;                  // the unit's state buffer and its phase
  // chunk i ^ (gtid % 8) of the thread's segment: eight threads' loads of 16
  // bytes then fall into different banks
  const uint32_t swz = static_cast<uint32_t>(gtid & 7);
  const uint8_t* const my_seg = ring + grp * kLpPieceBytes + 128 * gtid + 16 * swz;
  int kind = kind_of(first);
  for (int64_t u = first; u < units; u += G) {
    const int next = kind_of(u + G);
    if (kind <= 0) {
      kind = next;
      continue;
    }
    kind = next;
    const int nc_all = unit_chunks<ES>(a, u);
    const uint32_t np = static_cast<uint32_t>(nc_all + kLpPieceChunks - 1) / kLpPieceChunks;
    // the unit's states and keys go where unit k - 4's were
    bool ok = true;
    if (lane == 0) ok = wait(&sh.rowempty[j], jphase);
    if (!__all_sync(0xffffffffu, ok)) break;
    SoftState st{kNegInf, 0.0f, 0.0f};
    for (; turn < np; turn += kLpGroups) {
      const uint32_t s = gs * kLpGroups + grp;
      if (!__all_sync(0xffffffffu, wait(&sh.full[s], gphase))) {
        ok = false;
        break;
      }
      const uint8_t* seg = my_seg + gs * (kLpGroups * kLpPieceBytes);
      if (++gs == kGroupSlots) {
        gs = 0;
        gphase ^= 1;
      }
      const int nc = nc_all - static_cast<int>(turn) * kLpPieceChunks - kSegChunks * gtid;
      uint4 q[kSegChunks];
#pragma unroll
      for (int i = 0; i < kSegChunks; ++i)
        q[i] = *reinterpret_cast<const uint4*>(seg + (static_cast<int>((i ^ swz)) - static_cast<int>(swz)) * 16);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[s]);
      if (nc < kSegChunks) {  // a row's last piece: no chunks there
        const uint32_t none = ES == 2 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
        for (int i = 0; i < kSegChunks; ++i)
          if (static_cast<int>(i ^ swz) >= nc) q[i] = make_uint4(none, none, none, none);
      }
      if (nc > 0) {
        const float cm = fold_segment<T, ENT>(st, q, a.c, a.low);
        if constexpr (TOPK) seg_keys[j * a.seg_cap + turn * kPieceSegs + gtid] = order_key(cm);
      }
    }
    if (!ok) break;
    turn -= np;
    sh.part_rs[j][warp][lane] = make_float2(st.r, st.s);
    if constexpr (ENT) sh.part_t[j][warp][lane] = st.t;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.rowfull[j]);
    if (++j == kLpFinalizers) {
      j = 0;
      jphase ^= 1;
    }
  }
}

// Rows in slices: one warp per row merges the slices' states and alternatives.
constexpr int kMergeWarps = 4;

template <typename T>
__global__ void __launch_bounds__(32 * kMergeWarps) logprobs_merge_kernel(StatArgs a) {
  constexpr int ES = Elem<T>::kBytes;
  __shared__ uint64_t buf[kMergeWarps][kTopBuf], out[kMergeWarps][GH_MAX_TOP_K];
  pdl_wait();
  pdl_trigger();
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeWarps + warp; row < a.B;
       row += static_cast<int64_t>(gridDim.x) * kMergeWarps) {
    const int kind = row_kind(a, row);
    if (kind <= 0) {
      write_no_row(a.lp, row, kind);
      continue;
    }
    const uint8_t* src = static_cast<const uint8_t*>(a.logits) + row * a.ld * ES;
    const float xt = Elem<T>::load(src + a.lp.index[row] * ES);
    SoftState st{kNegInf, 0.0f, 0.0f};
    for (int i = lane; i < a.slices; i += 32) {
      const float4 v = a.part[row * a.slices + i];
      st = combine(st, SoftState{v.x, v.y, v.z});
    }
    st = warp_combine(st);
    WarpTopK top{buf[warp], out[warp], a.top_k, 0, 0};
    if (a.top_k > 0) {
      const uint64_t* keys = a.part_keys + row * a.slices * a.top_k;
      const int n = a.slices * a.top_k;
      for (int i = 0; i < n; i += 32) {
        const uint64_t key = i + lane < n ? keys[i + lane] : 0;
        top.push(key, key != 0);
      }
      top.cut();
    }
    write_row<T>(a.lp, row, row_dist<T>(st, src, a.V, a.c), xt, top.out);
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// Gradient of the row's log-probability and entropy, one read and one write of
// every logit:
//     grad_j = (1/T) (g_l [j == t] - p_j (g_l + g_H (log p_j + H))).
// With y = x c - lse log2(e),
//     grad_j = 2^y (a + b y) + [j == t] g_l / T,
//     a = -(g_l + g_H H) / T,  b = -g_H ln 2 / T.
// Logits with y < -512 give 0 in fp32; they are raised to about there, so that
// -inf gives 2^y (a + b y) = 0 as well.  The rounding of lse log2(e) moves to
// the factor 2^-lo of a and b; fp32 logits add the rounding of c.
//
// A CTA takes tiles of a row, four 16-byte chunks a thread; the row's scalars
// and the chunks are loaded together, so a tile waits for memory once.
// ---------------------------------------------------------------------------

// Beyond this |lse| its fp32 rounding (2^-14 here) would show in exp(x / T -
// lse): rows whose logits all lie far from 0, such as fully masked ones, have
// their max and sum taken again.
constexpr float kFarLse = 1024.0f;

constexpr int kVjpTileThreads = 256;
constexpr int kVjpTileUnroll = 4;
constexpr int kVjpTileChunks = kVjpTileThreads * kVjpTileUnroll;

constexpr float kLog2eLo = static_cast<float>(1.4426950408889634 - static_cast<double>(kLog2e));

struct VjpScalars {
  float sub, hi, a, b, gt, x0;
};

template <typename T>
__device__ __forceinline__ float vjp_element(float x, const VjpScalars& w, float c, float c_lo) {
  x = fmaxf(x - w.sub, w.x0);
  const float y = fmaf(x, c, Elem<T>::kBytes == 4 ? fmaf(x, c_lo, -w.hi) : -w.hi);
  return ex2(y) * fmaf(w.b, y, w.a);
}

template <typename T>
__device__ __forceinline__ void vjp_tile_chunk(const uint4& q, const VjpScalars& w, float c, float c_lo, int tj,
                                               uint8_t* dst, bool congruent) {
  constexpr int ES = Elem<T>::kBytes, EPC = 16 / ES;
  float v[EPC], g[EPC];
  unpack16<T>(q, v);
  const float2 c2 = make_float2(c, c), l2 = make_float2(c_lo, c_lo), h2 = make_float2(-w.hi, -w.hi),
               s2 = make_float2(-w.sub, -w.sub), a2 = make_float2(w.a, w.a), b2 = make_float2(w.b, w.b);
#pragma unroll
  for (int j = 0; j < EPC; j += 2) {
    float2 x = __fadd2_rn(make_float2(v[j], v[j + 1]), s2);
    x = make_float2(fmaxf(x.x, w.x0), fmaxf(x.y, w.x0));
    const float2 y = __ffma2_rn(x, c2, ES == 4 ? __ffma2_rn(x, l2, h2) : h2);
    const float2 r = __fmul2_rn(make_float2(ex2(y.x), ex2(y.y)), __ffma2_rn(b2, y, a2));
    g[j] = r.x;
    g[j + 1] = r.y;
  }
  if (tj >= 0) {
#pragma unroll
    for (int j = 0; j < EPC; ++j)
      if (j == tj) g[j] += w.gt;
  }
  if (congruent) {
    __stcs(reinterpret_cast<uint4*>(dst), pack16<T>(g));
  } else {
#pragma unroll
    for (int j = 0; j < EPC; ++j) Elem<T>::store(dst + j * ES, g[j]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kVjpTileThreads) logprobs_vjp_kernel(LogprobVjpArgs a, int64_t row_tiles) {
  constexpr int ES = Elem<T>::kBytes;
  __shared__ float red[2][kVjpTileThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = static_cast<int>(threadIdx.x);
  for (int64_t tile = blockIdx.x; tile < a.B * row_tiles; tile += gridDim.x) {
    const int64_t row = tile / row_tiles, part = tile - row * row_tiles;
    const RowGeo r = row_geo<ES>(a.logits, row, a.ld, a.V);
    const int64_t c0 = r.c_lo + part * kVjpTileChunks + tid;
    uint4 q[kVjpTileUnroll];
#pragma unroll
    for (int u = 0; u < kVjpTileUnroll; ++u) {
      const int64_t c = c0 + u * kVjpTileThreads;
      if (c < r.c_hi) q[u] = __ldcs(reinterpret_cast<const uint4*>(r.base + 16 * c));
    }
    const int64_t t = a.index[row];
    uint8_t* dst = static_cast<uint8_t*>(a.grad) + row * a.ld_grad * ES;
    uint8_t* gbase = dst - r.lead;  // chunk c's gradient bytes start at gbase + 16 c
    const bool congruent = ((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(r.src)) & 15) == 0;
    // the ragged ends go with the first tile, elements in lanes of its first warp
    const int64_t e = part == 0 && tid < 32 ? edge_element(r, a.V, tid) : -1;
    const float edge = e >= 0 ? Elem<T>::load(r.src + e * ES) : 0.0f;
    VjpScalars w{0.0f, 0.0f, 0.0f, 0.0f, 0.0f, kNegInf};
    const bool counts = t != a.ignore_index && t >= 0 && t < a.V;
    bool far = false;
    if (counts) {
      const float lse = a.lse[row], gl = a.g_logprob[row], gH = a.g_entropy ? a.g_entropy[row] : 0.0f;
      const float H = a.entropy[row];
      w.hi = lse * kLog2e;
      float lo = fmaf(lse, kLog2e, -w.hi) + lse * kLog2eLo;
      far = fabsf(lse) > kFarLse;
      if (far) {
        if (part != 0) continue;  // the row's first tile takes it whole (in place, its sums come before any store)
        float m = kNegInf, s = 0.0f;
        for (int64_t j = tid; j < a.V; j += kVjpTileThreads) m = fmaxf(m, Elem<T>::load(r.src + j * ES));
        m = block_max<kVjpTileThreads>(m, red[0]);
        for (int64_t j = tid; j < a.V; j += kVjpTileThreads) s += ex2((Elem<T>::load(r.src + j * ES) - m) * a.c);
        w.hi = log2f(block_sum<kVjpTileThreads>(s, red[1]));
        w.sub = m;
        lo = 0.0f;
        __syncthreads();
      }
      const float k = ex2(-lo);
      w.a = -(gl + gH * H) * a.inv_t * k;
      w.b = -gH * kLn2 * a.inv_t * k;
      w.gt = gl * a.inv_t;
      w.x0 = (w.hi - 512.0f) / a.c;
    } else if (tid == 0 && part == 0 && t != a.ignore_index) {
      record_status(GH_ERR_TARGET_RANGE);
    }
    if (counts) {
      const int64_t tb = r.lead + t * ES;
      const int64_t tc = tb >> 4;
      const int tj = static_cast<int>((tb & 15) / ES);
#pragma unroll
      for (int u = 0; u < kVjpTileUnroll; ++u) {
        const int64_t c = c0 + u * kVjpTileThreads;
        if (c < r.c_hi) vjp_tile_chunk<T>(q[u], w, a.c, a.c_lo, c == tc ? tj : -1, gbase + 16 * c, congruent);
      }
      if (far) {
        for (int64_t c = c0 + kVjpTileChunks; c < r.c_hi; c += kVjpTileThreads)
          vjp_tile_chunk<T>(__ldcs(reinterpret_cast<const uint4*>(r.base + 16 * c)), w, a.c, a.c_lo, c == tc ? tj : -1,
                            gbase + 16 * c, congruent);
      }
      if (e >= 0) Elem<T>::store(dst + e * ES, vjp_element<T>(edge, w, a.c, a.c_lo) + (e == t ? w.gt : 0.0f));
    } else {
#pragma unroll
      for (int u = 0; u < kVjpTileUnroll; ++u) {
        const int64_t c = c0 + u * kVjpTileThreads;
        if (c >= r.c_hi) break;
        if (congruent) {
          __stcs(reinterpret_cast<uint4*>(gbase + 16 * c), make_uint4(0, 0, 0, 0));
        } else {
          for (int j = 0; j < 16 / ES; ++j) Elem<T>::store(gbase + 16 * c + j * ES, 0.0f);
        }
      }
      if (e >= 0) Elem<T>::store(dst + e * ES, 0.0f);
    }
  }
}

int token_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n > 0 ? n : 148;
}

// Slices per row.  One unit costs its segments plus about 64 (a unit's fixed
// work), the merge about 850 (2.5 us at an SM's share of the copy rate); the
// busiest SM's total decides.  With alternatives a unit's keys fit shared memory.
int plan_slices(int64_t B, int64_t V, int es, bool topk, int sms) {
  const int64_t segs = (V * es + 16 * kSegChunks - 1) / (16 * kSegChunks) + 1;
  const int64_t lo = topk ? (segs + kLpMaxSegs - 1) / kLpMaxSegs : 1;
  const int64_t hi = tmax<int64_t>(lo, tmin<int64_t>(64, segs / kPieceSegs));
  int64_t best = lo, cost = INT64_MAX;
  for (int64_t s = lo; s <= hi; ++s) {
    const int64_t c = ((B * s + sms - 1) / sms) * ((segs + s - 1) / s + 64) + (s > 1 ? 850 : 0);
    if (c < cost) {
      cost = c;
      best = s;
    }
    if (B >= 64 * sms) break;
  }
  return static_cast<int>(best);
}

using StatKernel = void (*)(StatArgs);

template <bool ENT, bool TOPK>
StatKernel stat_kernel(int es) {
  return es == 4 ? static_cast<StatKernel>(logprobs_ring_kernel<float, ENT, TOPK>)
                 : static_cast<StatKernel>(logprobs_ring_kernel<uint16_t, ENT, TOPK>);
}

// The lowest logit that keeps x c finite, as packed bf16 or fp32 bits.
uint32_t low_bits(float c, int es) {
  const float low = -std::min(3.3e38f, 3.3e38f / c);
  uint32_t b;
  std::memcpy(&b, &low, 4);
  return es == 4 ? b : (b >> 16) * 0x10001u;  // truncated towards 0
}

}  // namespace

gh_status_t logprobs_launch(const LogprobArgs& o, gh_dtype_t dtype, cudaStream_t stream) {
  const int es = dtype == GH_F32 ? 4 : 2;
  const bool topk = o.top_k > 0;
  const int sms = token_sm_count();
  StatArgs a{};
  a.logits = o.logits;
  a.B = o.B;
  a.V = o.V;
  a.ld = o.ld;
  a.c = o.c;
  a.low = low_bits(o.c, es);
  a.top_k = o.top_k;
  a.lp = o;
  a.slices = plan_slices(o.B, o.V, es, topk, sms);
  const int64_t segs = (o.V * es + 127) / 128 + 1;
  a.slice_segs = static_cast<int>((segs + a.slices - 1) / a.slices);
  a.seg_cap = (a.slice_segs + 127) / 128 * 128;
  const int64_t units = o.B * a.slices;

  void* scratch = nullptr;
  if (a.slices > 1) {
    const gh_status_t st = scratch_alloc(&scratch, static_cast<size_t>(units) * (16 + 8 * o.top_k), stream);
    if (st != GH_OK) return st;
    a.part = static_cast<float4*>(scratch);
    a.part_keys = reinterpret_cast<uint64_t*>(static_cast<char*>(scratch) + units * 16);
  }
  const StatKernel kern = topk ? stat_kernel<true, true>(es) : stat_kernel<true, false>(es);
  const int smem = topk ? lp_smem_bytes<true>(a.seg_cap) : lp_smem_bytes<false>(0);
  gh_status_t st = ensure_smem_limit(kern, topk ? lp_smem_bytes<true>(kLpMaxSegs) : smem) == cudaSuccess ? GH_OK : GH_ERR_CUDA;
  if (st == GH_OK) {
    ProfileScope prof(GH_KERNEL_LOGPROBS, stream);
    note_launch();
    if (launch_pdl(kern, dim3(static_cast<unsigned>(tmin<int64_t>(units, sms))), dim3(kLpThreads), smem, stream, 1, a) !=
        cudaSuccess)
      st = GH_ERR_CUDA;
    if (st == GH_OK && a.slices > 1) {
      const unsigned grid = static_cast<unsigned>(tmin<int64_t>((o.B + kMergeWarps - 1) / kMergeWarps, 8 * sms));
      note_launch();
      const StatKernel merge = es == 4 ? static_cast<StatKernel>(logprobs_merge_kernel<float>)
                                       : static_cast<StatKernel>(logprobs_merge_kernel<uint16_t>);
      if (launch_pdl(merge, dim3(grid), dim3(32 * kMergeWarps), 0, stream, 1, a) != cudaSuccess) st = GH_ERR_CUDA;
    }
  }
  scratch_free(scratch, stream);
  return st;
}

gh_status_t logprobs_vjp_launch(const LogprobVjpArgs& a, gh_dtype_t dtype, cudaStream_t stream) {
  const int es = dtype == GH_F32 ? 4 : 2;
  const int64_t row_tiles = tmax<int64_t>(1, (a.V * es / 16 + kVjpTileChunks - 1) / kVjpTileChunks);
  const unsigned grid = static_cast<unsigned>(tmin<int64_t>(a.B * row_tiles, static_cast<int64_t>(token_sm_count()) * 8));
  ProfileScope prof(GH_KERNEL_LOGPROBS_VJP, stream);
  note_launch();
  const cudaError_t e =
      dtype == GH_F32
          ? launch_pdl(logprobs_vjp_kernel<float>, dim3(grid), dim3(kVjpTileThreads), 0, stream, 1, a, row_tiles)
          : launch_pdl(logprobs_vjp_kernel<uint16_t>, dim3(grid), dim3(kVjpTileThreads), 0, stream, 1, a, row_tiles);
  return e == cudaSuccess ? GH_OK : GH_ERR_CUDA;
}

}  // namespace gh
