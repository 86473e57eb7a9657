// Log-probabilities of given tokens with the row's entropy, log-sum-exp and
// most probable alternatives, and their gradient.
//
// For a row x of V logits, temperature T and c = log2(e) / T, with a reference
// R near its largest x c,
//     y_j = x_j c - R,   s = sum_j 2^y_j,   t = sum_j 2^y_j y_j,   y_m = M c - R,
//     l = log sum_j exp((x_j - M) / T) = log1p((s - 2^y_m) 2^-y_m),
//     log p_j = (x_j - M) / T - l,   lse = M / T + l,
//     entropy = l - ln 2 (t / s - y_m)
// (a term with 2^y = 0 adds nothing to t, so -inf logits are 0 log 0 = 0).
// The alternatives are the top_k logits by (value descending, index
// ascending); the temperature does not change their order.
//
// The forward (logprobs_kernel) reads every logit once.  A row is cut into
// segments (512 bytes, one 16-byte load of a warp; finer ones for short rows),
// and the key of each segment's largest logit is kept in shared memory.  The k
// largest logits lie in the k segments that come first by (largest logit
// descending, position ascending): any other segment's logits have k segment
// maxima before them.  So the alternatives cost a maximum per segment during the
// pass, a selection among V / 256 (bf16) keys, and k segments read again from L2.
#include <algorithm>
#include <cstring>

#include "profile.h"
#include "threshold_search.h"
#include "token_device.cuh"
#include "token_ops.h"

namespace gh {

namespace {

// ---------------------------------------------------------------------------
// Forward.  One CTA of four warps per row, seven or eight of them on an SM, so
// that one's end (merge, alternatives) overlaps the others' streams.  The warps
// take batches of four segments in turn, the next batch's loads in flight while
// one is summed.  Small batches and very long rows take a cluster of up to eight
// CTAs per row, whose first merges the others' sums and alternatives through
// distributed shared memory.
//
// Bound by HBM where no alternatives are asked for: [4096, 50257] fp32 in 120
// us (6.8 TB/s), [8192, 50257] bf16 in 125 us from a cool start (6.5 TB/s) and
// 131 to 148 under the power cap, with the special-function unit 67% busy.  With
// alternatives the segments' maxima (41 warp instructions more a batch of 2 KiB a
// warp, on 176) and the row's end (2,500 with 20 alternatives) add instructions,
// and at the end one warp picks segments while others wait (barrier stalls 1.1 per
// issue; no unit is full, issue slots 55%): [4096, 50257] bf16 with 32 in 90 to 96
// us, [1024, 262144] with 128 in 107 to 120, [4096, 50257] fp32 with 32 in 147 to 155.
//
// Warps per CTA, on one board in turn, at [8192, 50257] bf16 / [1024, 262144] bf16
// / [4096, 50257] fp32 without alternatives, and with 32 / 128 / 32: 4 139 / 110 /
// 123 and 189 / 120 / 158 us, 2 141 / 124 / 123 and 180 / 216 / 199, 8 150 / 93 / 123 and
// 242 / 126 / 183; 4 and a CTA more per SM with alternatives (64 registers for 72)
// 193 / 143 / 162.  At 72 registers the fp32 kernels with alternatives and the bf16
// one of split rows with finer segments spill 4 to 40 bytes a thread.
// ---------------------------------------------------------------------------

constexpr int kLpWarps = 4;
// Rows of up to 16 KiB take CTAs of one warp once there are more of them than
// CTAs of four are resident: the fixed work of a row's end is then one warp's
// ([4750, 1204] bf16 with 2 alternatives 23.7 -> 14.0 us, [4000, 8192] with 20
// 30.5 -> 25.9; 32 KiB rows lose: [2000, 16384] 21.1 -> 28.8).
constexpr int64_t kShortChunks = 1024;
constexpr int kMaxSlices = 8;       // CTAs per row: a portable cluster
constexpr int kLpMaxSegs = 16384;   // 512-byte segments of a CTA whose keys are kept (64 KiB)

// How many logits of the picked segments may reach the threshold, and chunks
// have one, before the slow way.
template <int W>
constexpr int kCandidates = W == 1 ? 256 : 512;
template <int W>
constexpr int kHitChunks = W == 1 ? 192 : 256;

// Segments: a warp's load (512 bytes), four lanes' (64), one lane's (16), or one
// logit.  The finer ones are for rows with few segments per alternative.
enum SegKind : int { kSegElement = 0, kSegChunk = 1, kSegQuad = 2, kSegWarp = 3 };
// What a kernel keeps for alternatives: nothing, warp segments' keys, or finer ones'.
enum TopMode : int { kTopNone = 0, kTopWarp = 1, kTopFine = 2 };

// How many segments may be listed for k alternatives.  A few more than k end the
// search for a threshold sooner: [1, 50257] bf16 with 20 alternatives 10.9 -> 9.9
// us, [214, 22627] fp32 with 36 17.8 -> 16.1, [2701, 3400] fp32 with 107 32.6 ->
// 31.4; many more would cost more ranking.
__host__ __device__ constexpr int most_listed(int k) { return k + k / 8 + 2; }

template <int W>
struct LpShared {
  LaneSums<W, true> sums;
  float4 part;  // this CTA's (maximum, reference, sum, weighted sum), read by the cluster's first
  RowDist dist;
  int count, chunks, listed;
  float least;
  int list[most_listed(GH_MAX_TOP_K)];
};
template <int W>
struct LpTopShared {
  uint64_t buf[kCandidates<W>];
  uint64_t out[GH_MAX_TOP_K];  // this CTA's alternatives, largest first, zeros behind them
  uint4 hit[kHitChunks<W>];    // chunks with a candidate, and which they are
  int hit_chunk[kHitChunks<W>];
};
static_assert(kMaxSlices * GH_MAX_TOP_K <= 1024, "the keys gathered by a cluster's first CTA");
static_assert(kCandidates<1> >= kTopBuf && kCandidates<kLpWarps> >= kTopBuf, "the slow way's buffer");

// Rows that count: 1; ignored: 0; an index outside [0, V): -1.
__device__ __forceinline__ int row_kind(const LogprobArgs& a, int64_t row) {
  const int64_t t = a.index[row];
  if (t == a.ignore_index) return 0;
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

// One alternative of a row.
__device__ __forceinline__ void write_top(const LogprobArgs& o, int64_t row, const RowDist& d, int k, uint64_t key) {
  o.top_logprob[row * o.top_k + k] = d.none ? kNaN : log_p(d, key_value(key), o.temperature);
  o.top_index[row * o.top_k + k] = d.none ? -1 : key_index(key);
}

// Values of a row that counts (by one thread).
__device__ __forceinline__ void write_values(const LogprobArgs& o, int64_t row, const RowDist& d, float xt) {
  o.logprob[row] = d.none ? kNaN : log_p(d, xt, o.temperature);
  o.entropy[row] = d.none ? kNaN : d.entropy;
  o.lse[row] = d.none ? kNaN : d.m / o.temperature + d.l;
}

// A warp's keys in registers: lane l has keys l, l + 32, ... (zeros behind the last).
template <int R>
struct LaneKeys {
  uint32_t v[R];
  __device__ __forceinline__ void load(const uint32_t* keys, int segs) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = 32 * i + lane < segs ? keys[32 * i + lane] : 0;
  }
  // how many of the warp's keys are >= c
  __device__ __forceinline__ int count(uint32_t c) const {
    int n[4] = {};  // (short chains)
#pragma unroll
    for (int i = 0; i < R; ++i) n[i % 4] += v[i] >= c ? 1 : 0;
    return __reduce_add_sync(0xffffffffu, n[0] + n[1] + (n[2] + n[3]));
  }
  __device__ __forceinline__ uint32_t lane_max() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) m = max(m, v[i]);
    return m;
  }
  // positions of the keys >= c; returns how many
  __device__ __forceinline__ int list_from(uint32_t c, int* list) const {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    int n = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint32_t got = __ballot_sync(0xffffffffu, v[i] >= c);
      if (v[i] >= c) list[n + __popc(got & ((1u << lane) - 1))] = 32 * i + lane;
      n += __popc(got);
    }
    return n;
  }
};

// The same over keys left in shared memory.
template <>
struct LaneKeys<0> {
  const uint32_t* keys;
  int segs;
  __device__ __forceinline__ void load(const uint32_t* from, int n) {
    keys = from;
    segs = n;
  }
  __device__ __forceinline__ int count(uint32_t c) const {
    // (four at a time: zeros fill the keys up to a multiple of 128)
    const uint4* k4 = reinterpret_cast<const uint4*>(keys);
    int n = 0;
    for (int i = static_cast<int>(threadIdx.x) & 31; 4 * i < segs; i += 32)
      n += (k4[i].x >= c) + (k4[i].y >= c) + (k4[i].z >= c) + (k4[i].w >= c);
    return __reduce_add_sync(0xffffffffu, n);
  }
  __device__ __forceinline__ uint32_t lane_max() const {
    uint32_t m = 0;
    for (int i = static_cast<int>(threadIdx.x) & 31; i < segs; i += 32) m = max(m, keys[i]);
    return m;
  }
  __device__ __forceinline__ int list_from(uint32_t c, int* list) const {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    int n = 0;
    for (int i = 0; i < segs; i += 32) {
      const bool take = i + lane < segs && keys[i + lane] >= c;
      const uint32_t got = __ballot_sync(0xffffffffu, take);
      if (take) list[n + __popc(got & ((1u << lane) - 1))] = i + lane;
      n += __popc(got);
    }
    return n;
  }
};

static_assert(most_listed(GH_MAX_TOP_K) < 256, "the zeros behind the keys are never listed");

// search_threshold by one warp, in units of 2^kShift (bf16 keys differ in their
// upper 16 bits only): between the least of the lanes' largest keys, which 32
// keys reach, and the largest.
template <typename T, int R>
__device__ __forceinline__ uint32_t kth_key(const LaneKeys<R>& keys, int k, bool* found) {
  constexpr int kShift = Elem<T>::kBytes == 2 ? 16 : 0;
  const uint32_t m = keys.lane_max();
  const uint32_t hi = __reduce_max_sync(0xffffffffu, m) >> kShift, lo = __reduce_min_sync(0xffffffffu, m) >> kShift;
  return search_threshold(lo, hi, k, most_listed(k), [&](uint32_t v) { return keys.count(v << kShift); }, found) << kShift;
}

// Segments that hold the k largest logits, of `segs` with these keys (padded with
// zeros to a multiple of 128), by one warp: all that reach a key that k of them
// reach, or the first k by (key descending, position ascending).  Their
// positions go into list[], in order; returns how many (at most most_listed(k)),
// and in thr a key that k of all the logits reach (0: all are listed).
template <typename T, int R>
__device__ __forceinline__ int pick_from(const uint32_t* keys, int segs, int k, int* list, uint32_t* thr) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  LaneKeys<R> v;
  v.load(keys, segs);
  bool found;
  const uint32_t key = kth_key<T, R>(v, k, &found);
  *thr = key;
  if (found) return v.list_from(key, list);
  // Some keys tie at the k-th: all above it, and the first of the equal ones.
  // (A negative bf16 value's key ends in ones: compare the kept bits.)
  const uint32_t mask = Elem<T>::kBytes == 2 ? 0xffff0000u : 0xffffffffu;
  const uint32_t below = (1u << lane) - 1;
  int above = 0, n = 0;
  for (int i = lane; i < segs; i += 32) above += (keys[i] & mask) > key;
  int left = k - __reduce_add_sync(0xffffffffu, above);
  for (int i = 0; i < segs && n < k; i += 32) {
    const uint32_t q = i + lane < segs ? keys[i + lane] & mask : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, q == key);
    const bool take = q > key || (q == key && __popc(eq & below) < left);
    const uint32_t got = __ballot_sync(0xffffffffu, take);
    if (take) list[n + __popc(got & below)] = i + lane;
    n += __popc(got);
    left -= tmin(left, __popc(eq));
  }
  return n;
}

template <typename T>
__device__ __forceinline__ int pick_segments(const uint32_t* keys, int segs, int k, int* list, uint32_t* thr) {
  // (fewer segments than that: a key below every logit's could be found)
  if (segs <= most_listed(k)) {
    for (int i = static_cast<int>(threadIdx.x) & 31; i < segs; i += 32) list[i] = i;
    *thr = 0;
    return segs;
  }
  return segs <= 256    ? pick_from<T, 8>(keys, segs, k, list, thr)
         : segs <= 1024 ? pick_from<T, 32>(keys, segs, k, list, thr)
                        : pick_from<T, 0>(keys, segs, k, list, thr);
}

// A threshold key as a logit: keys at or above it are logits >= it.
template <typename T>
__device__ __forceinline__ float least_of(uint32_t thr) {
  if (thr == 0) return kNegInf;
  if (Elem<T>::kBytes == 2 && !(thr & 0x80000000u)) thr |= 0xffffu;  // the bf16 value itself
  return key_value(static_cast<uint64_t>(thr) << 32);
}

__device__ __forceinline__ uint64_t ld_dsmem_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// A CTA's part of a row: its first chunk, how many, that chunk's first element's
// index in the row, and the chunks of a segment (2^shift).
struct RowPart {
  const uint4* chunks;
  int64_t j0;
  int nc, shift;
};

// Loads, by one warp, the chunks of the 32 >> shift listed segments from place
// `at` on: a lane's chunk of the part (nc: none).
__device__ __forceinline__ int listed_chunk(RowPart w, const int* list, int n, int at) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  at += lane >> w.shift;
  return at < n ? (list[at] << w.shift) + (lane & ((1 << w.shift) - 1)) : w.nc;
}

// The k largest keys of the listed segments and the ragged ends, by one warp
// and whatever their number (ties can make it large): into out[]; returns how many.
template <typename T>
__device__ __noinline__ int pick_slowly(uint64_t* buf, uint64_t* out, RowPart w, const int* list, int n, int k,
                                        float edge, int64_t e) {
  constexpr int EPC = 16 / Elem<T>::kBytes;
  WarpTopK top{buf, out, k, 0, 0};
  for (int at = 0; at < n; at += 32 >> w.shift) {
    const int c = listed_chunk(w, list, n, at);
    const uint4 q = c < w.nc ? __ldcg(w.chunks + c) : make_uint4(0, 0, 0, 0);
    float v[EPC];
    unpack16<T>(q, v);
#pragma unroll
    for (int j = 0; j < EPC; ++j) top.push(rank_key(order_key(v[j]), w.j0 + static_cast<int64_t>(c) * EPC + j), c < w.nc);
  }
  top.push(rank_key(order_key(edge), e), e >= 0);
  top.cut();
  return top.n;
}

// CTAs of W warps on an SM (W == 1: as many as 80 registers a thread allow).
template <int TOP, int W>
constexpr int kLpResident = W == 1 ? (TOP != kTopNone ? 21 : 24) : (TOP != kTopNone ? 7 : 8);

template <typename T, int TOP, bool SPLIT, int W>
__global__ void __launch_bounds__(32 * W, kLpResident<TOP, W>) logprobs_kernel(LogprobArgs a) {
  constexpr int kThreads = 32 * W;
  constexpr int ES = Elem<T>::kBytes, EPC = 16 / ES;
  __shared__ LpShared<W> sh;
  __shared__ LpTopShared<W> tsh;
  extern __shared__ __align__(16) float seg_max[];  // the segments' largest logits; their keys once picked from
  uint32_t* const seg_keys = reinterpret_cast<uint32_t*>(seg_max);
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const int tid = static_cast<int>(threadIdx.x);
  pdl_wait();
  pdl_trigger();
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t row = SPLIT ? blockIdx.x / a.slices : blockIdx.x;
  const bool last = !SPLIT || rank == a.slices - 1;
  const RowGeo r = row_geo<ES>(a.logits, row, a.ld, a.V);
  const int64_t from = SPLIT ? tmin(r.c_hi, r.c_lo + rank * a.slice_chunks) : r.c_lo;
  const int nc = static_cast<int>((last ? r.c_hi : tmin(r.c_hi, from + a.slice_chunks)) - from);
  const uint4* const chunks = reinterpret_cast<const uint4*>(r.base) + from + lane;
  const uint32_t none = ES == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
  auto load = [&](uint4 (&q)[kBatch], int c0) {  // c0: the batch's first chunk of the part
    if (c0 + kBatchChunks <= nc) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) q[i] = __ldcg(chunks + c0 + i * kSegChunks);
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        q[i] = make_uint4(none, none, none, none);
        if (c0 + i * kSegChunks + lane < nc) q[i] = __ldcg(chunks + c0 + i * kSegChunks);
      }
    }
  };
  // the first loads start before it is known whether the row counts
  uint4 qa[kBatch], qb[kBatch];
  int c0 = warp * kBatchChunks;
  load(qa, c0);
  const int kind = row_kind(a, row);
  if (kind <= 0) {  // (the same in every CTA of a cluster)
    if (rank == 0 && warp == 0) write_no_row(a, row, kind);
    return;
  }
  // the last warp takes the ragged ends, and with them the row's values
  constexpr int kEnds = W - 1;
  int64_t e = -1;
  float edge = kNegInf, xt = 0.0f;
  if (warp == kEnds) {
    e = edge_element(r, a.V, lane);
    if (lane < 16 ? rank != 0 : !last) e = -1;
    if (e >= 0) edge = Elem<T>::load(r.src + e * ES);
    if (rank == 0) xt = Elem<T>::load(r.src + a.index[row] * ES);
  }

  WarpSums sums{kNegInf, kNegInf, {}, {}};
  auto fold = [&](const uint4 (&q)[kBatch], int c0) {
    float m[kBatch];
    fold_batch<T, true, TOP == kTopWarp>(sums, q, a.c, a.low, m);
    if constexpr (TOP == kTopWarp) {
      static_assert(kBatch == 4, "a batch's segments are stored together");
      if (lane == 0) *reinterpret_cast<float4*>(seg_max + c0 / kSegChunks) = make_float4(m[0], m[1], m[2], m[3]);
    }
    if constexpr (TOP == kTopFine) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + i * kSegChunks + lane;
        if (a.seg_kind == kSegElement) {
          float v[EPC];
          unpack16<T>(q[i], v);
#pragma unroll
          for (int j = 0; j < EPC; ++j) seg_max[c * EPC + j] = v[j];
          continue;
        }
        float v = max_of4<T>(q[i]);
        if (a.seg_kind == kSegQuad) {
          v = f32_max_nan(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = f32_max_nan(v, __shfl_xor_sync(0xffffffffu, v, 2));
          if ((lane & 3) == 0) seg_max[c >> 2] = v;
        } else {
          seg_max[c] = v;
        }
      }
    }
  };
  constexpr int kStep = W * kBatchChunks;
  while (c0 < nc) {
    if (c0 + kStep < nc) load(qb, c0 + kStep);
    fold(qa, c0);
    c0 += kStep;
    if (c0 >= nc) break;
    if (c0 + kStep < nc) load(qa, c0 + kStep);
    fold(qb, c0);
    c0 += kStep;
  }
  if (warp == kEnds) fold_lanes<true>(sums, edge, a.c);
  sh.sums.post(warp, lane, sums);
  if (TOP != kTopNone && tid == 0) sh.count = sh.chunks = 0;
  __syncthreads();

  // the last warp merges the sums while warp 0 picks the segments
  const RowPart part{chunks - lane, (16 * from - r.lead) / ES, nc,
                     TOP == kTopWarp || a.seg_kind == kSegWarp ? 5 : a.seg_kind == kSegQuad ? 2 : 0};
  const bool elements = TOP == kTopFine && a.seg_kind == kSegElement;
  if (TOP != kTopNone && warp == 0) {
    const int segs = elements ? nc * EPC : (nc + (1 << part.shift) - 1) >> part.shift;
    // keys, zeros up to a multiple of 128
    uint4* const k4 = reinterpret_cast<uint4*>(seg_keys);
    for (int j = lane; j < (segs + 127) / 128 * 32; j += 32) {
      const float4 v = reinterpret_cast<const float4*>(seg_max)[j];
      k4[j] = make_uint4(4 * j < segs ? order_key(v.x) : 0u, 4 * j + 1 < segs ? order_key(v.y) : 0u,
                         4 * j + 2 < segs ? order_key(v.z) : 0u, 4 * j + 3 < segs ? order_key(v.w) : 0u);
    }
    __syncwarp();
    uint32_t thr;
    const int n = pick_segments<T>(seg_keys, segs, a.top_k, sh.list, &thr);
    if (lane == 0) {
      sh.listed = n;
      sh.least = least_of<T>(thr);
    }
  }
  if (warp == kEnds) {
    const SoftState all = sh.sums.merge(lane);
    if (SPLIT) {
      if (lane == 0) sh.part = make_float4(all.m, all.r, all.s, all.t);
    } else {
      const RowDist d = row_dist<T>(all, r.src, a.V, a.c);
      if (lane == 0) {
        write_values(a, row, d, xt);
        if (TOP != kTopNone) sh.dist = d;
      }
    }
  }
  int n = 0;
  if constexpr (TOP != kTopNone) {
    __syncthreads();
    // every logit of the picked segments that reaches the threshold is a candidate
    const int listed = sh.listed;
    const float least = sh.least;
    auto offer = [&](float x, int64_t j) {
      const int p = atomicAdd(&sh.count, 1);
      if (p < kCandidates<W>) tsh.buf[p] = rank_key(order_key(x), j);
    };
    if (elements) {
      for (int i = tid; i < listed; i += kThreads) {
        const int at = sh.list[i];
        offer(key_value(static_cast<uint64_t>(seg_keys[at]) << 32), part.j0 + at);
      }
    } else {
      constexpr int kAhead = 8;
      const int per = 32 >> part.shift;  // segments of a warp's load
      for (int i0 = warp * per; i0 < listed; i0 += W * kAhead * per) {
        uint4 q[kAhead];
        int c[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          c[i] = listed_chunk(part, sh.list, listed, i0 + i * W * per);
          if (c[i] < nc) q[i] = __ldcg(part.chunks + c[i]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (c[i] >= nc || !(max_of4<T>(q[i]) >= least)) continue;
          const int p = atomicAdd(&sh.chunks, 1);
          if (p < kHitChunks<W>) {
            tsh.hit[p] = q[i];
            tsh.hit_chunk[p] = c[i];
          }
        }
      }
      __syncthreads();
      // (few lanes of a warp have such a chunk: one a thread from here)
      const int chunks_hit = sh.chunks;
      for (int i = tid; i < tmin(chunks_hit, kHitChunks<W>); i += kThreads) {
        float v[EPC];
        unpack16<T>(tsh.hit[i], v);
        const int64_t j0 = part.j0 + static_cast<int64_t>(tsh.hit_chunk[i]) * EPC;
#pragma unroll
        for (int j = 0; j < EPC; ++j)
          if (v[j] >= least) offer(v[j], j0 + j);
      }
      if (tid == 0 && chunks_hit > kHitChunks<W>) atomicAdd(&sh.count, kCandidates<W> + 1);  // the slow way
    }
    if (e >= 0 && edge >= least) offer(edge, e);
    __syncthreads();
    n = sh.count;
    if (n > kCandidates<W>) {  // the same n in every thread
      __syncthreads();
      if (warp == kEnds) {
        n = pick_slowly<T>(tsh.buf, tsh.out, part, sh.list, listed, a.top_k, edge, e);
        if (lane == 0) sh.count = n;
      }
      __syncthreads();
      n = sh.count;
    }
    // Each candidate's place is the number of larger ones (keys are distinct, so
    // the order of the offers does not matter).  A part, or a row without a
    // distribution, may have fewer than top_k.
    const RowDist d = sh.dist;
    auto put = [&](int place, uint64_t key) {
      if (SPLIT) tsh.out[place] = key;
      else write_top(a, row, d, place, key);
    };
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = tsh.buf[i];
      int above = 0;
      for (int j = 0; j < n; ++j) above += tsh.buf[j] > key ? 1 : 0;
      if (above < a.top_k) put(above, key);
    }
    for (int i = tmin(n, a.top_k) + tid; i < a.top_k; i += kThreads) put(i, 0);
  }
  if constexpr (SPLIT) {
    // the cluster's first CTA merges the parts
    __syncwarp();
    cluster_arrive_release();
    cluster_wait_acquire();
    if (rank == 0) {
      if (warp == kEnds) {
        SoftState all = kNoState;
        for (int i = 0; i < a.slices; ++i) {
          const uint32_t p = map_to_rank(&sh.part, i);
          all = combine(all, SoftState{ld_dsmem_f32(p), ld_dsmem_f32(p + 4), ld_dsmem_f32(p + 8), ld_dsmem_f32(p + 12)});
        }
        const RowDist d = row_dist<T>(all, r.src, a.V, a.c);
        if (lane == 0) {
          write_values(a, row, d, xt);
          sh.dist = d;
        }
      }
      if constexpr (TOP != kTopNone) {
        // The parts' alternatives in the row's order, then as logits of a row whose
        // segments are single logits; up to 64 are all ranked ([142, 167081] bf16
        // with 4 alternatives 23.6 -> 22.0 us; at 80, [1, 50257] with 10, both take 9.1).
        const int total = a.slices * a.top_k;
        const bool pick = total > 64;
        uint64_t* const gathered = reinterpret_cast<uint64_t*>(seg_keys + (total + 127) / 128 * 128);
        for (int i = tid; i < (total + 127) / 128 * 128; i += kThreads) {
          uint64_t key = 0;
          if (i < total) {
            key = ld_dsmem_u64(map_to_rank(&tsh.out[i % a.top_k], i / a.top_k));
            gathered[i] = key;
          }
          seg_keys[i] = static_cast<uint32_t>(key >> 32);
        }
        __syncthreads();
        if (pick) {
          if (warp == 0) {
            uint32_t thr;
            const int got = pick_segments<T>(seg_keys, total, a.top_k, sh.list, &thr);
            if (lane == 0) sh.listed = got;
          }
          __syncthreads();
        }
        // (a row without a distribution may have too few alternatives for its places)
        const RowDist d = sh.dist;
        for (int i = tid; d.none && i < a.top_k; i += kThreads) write_top(a, row, d, i, 0);
        const int got = d.none ? 0 : pick ? sh.listed : total;
        for (int i = tid; i < got; i += kThreads) {
          const uint64_t key = gathered[pick ? sh.list[i] : i];
          int above = 0;
          for (int j = 0; j < got; ++j) above += gathered[pick ? sh.list[j] : j] > key ? 1 : 0;
          if (above < a.top_k) write_top(a, row, d, above, key);
        }
      }
    }
    // no CTA leaves before its part has been read
    __syncwarp();
    cluster_arrive_release();
    cluster_wait_acquire();
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
// One CTA of four warps per part of a row (parts of about 32 KiB), eight on an
// SM; the warps stream batches as the forward does.  Bound by HBM: [8192, 50257]
// bf16 in 246 to 268 us and [1024, 128256] fp32 in 158 to 170, both at the copy rate
// (the bf16 kernel spills 28 bytes a thread at 64 registers).  The parts' size
// matters because the CTAs in flight then read and write one stretch of memory:
// [8192, 50257] bf16 / [4096, 50257] fp32 249 / 246 us, with parts of 16 KiB 256 / 243,
// of 64 KiB 259 / 253.
// ---------------------------------------------------------------------------

// Beyond this |lse| its fp32 rounding (2^-14 here) would show in exp(x / T -
// lse): rows whose logits all lie far from 0, such as fully masked ones, and
// ordinary ones at low temperatures (logits near 10 from T = 0.01 down) have their
// max and sum taken again, by the CTA of their first part alone: [8192, 50257] bf16
// 704 us where every row is one, 249 otherwise.
constexpr float kFarLse = 1024.0f;

constexpr int kLpVjpWarps = 4;
constexpr int kLpVjpThreads = 32 * kLpVjpWarps;
constexpr int64_t kVjpPartBytes = 32 * 1024;

constexpr float kLog2eLo = static_cast<float>(1.4426950408889634 - static_cast<double>(kLog2e));

struct VjpScalars {
  float sub, hi, a, b, gt, x0;
};

// FAR: rows with sub != 0.
template <typename T, bool FAR>
__device__ __forceinline__ float vjp_element(float x, const VjpScalars& w, float c, float c_lo) {
  x = fmaxf(FAR ? x - w.sub : x, w.x0);
  const float y = fmaf(x, c, Elem<T>::kBytes == 4 ? fmaf(x, c_lo, -w.hi) : -w.hi);
  return ex2(y) * fmaf(w.b, y, w.a);
}

template <typename T, bool FAR>
__device__ __forceinline__ void lp_vjp_chunk(uint4 q, const VjpScalars& w, uint32_t low, float c, float c_lo, int tj,
                                          uint8_t* dst, bool congruent) {
  constexpr int ES = Elem<T>::kBytes, EPC = 16 / ES;
  if (!FAR) q = clamp_low<T>(q, low);
  float v[EPC], g[EPC];
  unpack16<T>(q, v);
  const float2 c2 = make_float2(c, c), l2 = make_float2(c_lo, c_lo), h2 = make_float2(-w.hi, -w.hi),
               a2 = make_float2(w.a, w.a), b2 = make_float2(w.b, w.b);
#pragma unroll
  for (int j = 0; j < EPC; j += 2) {
    float2 x = make_float2(v[j], v[j + 1]);
    if (FAR) x = make_float2(fmaxf(x.x - w.sub, w.x0), fmaxf(x.y - w.sub, w.x0));
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
__global__ void __launch_bounds__(kLpVjpThreads, 8) logprobs_vjp_kernel(LogprobVjpArgs a) {
  constexpr int ES = Elem<T>::kBytes;
  __shared__ float red[2][kLpVjpWarps];
  pdl_wait();
  pdl_trigger();
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int64_t row = a.parts == 1 ? blockIdx.x : blockIdx.x / a.parts;
  const int part = static_cast<int>(blockIdx.x - row * a.parts);
  const RowGeo r = row_geo<ES>(a.logits, row, a.ld, a.V);
  const int64_t from = tmin(r.c_hi, r.c_lo + part * a.part_chunks);
  int64_t nc = (part == a.parts - 1 ? r.c_hi : tmin(r.c_hi, from + a.part_chunks)) - from;
  const uint4* const chunks = reinterpret_cast<const uint4*>(r.base) + from + lane;
  constexpr int kStep = kLpVjpWarps * kBatchChunks;
  auto load = [&](uint4 (&q)[kBatch], int64_t c0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c0 + i * kSegChunks + lane < nc) q[i] = __ldcs(chunks + c0 + i * kSegChunks);
  };
  uint4 qa[kBatch], qb[kBatch];
  int64_t c0 = warp * kBatchChunks;
  load(qa, c0);
  const int64_t t = a.index[row];
  const bool counts = t != a.ignore_index && t >= 0 && t < a.V;
  uint8_t* const dst = static_cast<uint8_t*>(a.grad) + row * a.ld_grad * ES;
  uint8_t* const gbase = dst - r.lead + 16 * from;  // this part's chunk c's gradient starts at gbase + 16 c
  const bool congruent = ((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(r.src)) & 15) == 0;
  // the ragged ends go with the first part, elements in lanes of its first warp
  const int64_t e = part == 0 && warp == 0 ? edge_element(r, a.V, lane) : -1;
  const float edge = e >= 0 ? Elem<T>::load(r.src + e * ES) : 0.0f;
  if (!counts) {
    if (tid == 0 && part == 0 && t != a.ignore_index) record_status(GH_ERR_TARGET_RANGE);
    for (int64_t c = tid; c < nc; c += kLpVjpThreads) {
      if (congruent) {
        __stcs(reinterpret_cast<uint4*>(gbase + 16 * c), make_uint4(0, 0, 0, 0));
      } else {
        for (int j = 0; j < 16 / ES; ++j) Elem<T>::store(gbase + 16 * c + j * ES, 0.0f);
      }
    }
    if (e >= 0) Elem<T>::store(dst + e * ES, 0.0f);
    return;
  }
  VjpScalars w;
  const float lse = a.lse[row], gl = a.g_logprob[row], gH = a.g_entropy ? a.g_entropy[row] : 0.0f;
  const float H = a.entropy[row];
  w.hi = lse * kLog2e;
  w.sub = 0.0f;
  float lo = fmaf(lse, kLog2e, -w.hi) + lse * kLog2eLo;
  const bool far = fabsf(lse) > kFarLse;
  if (far) {
    // the row's first part takes it whole (in place, its sums come before any store)
    if (part != 0) return;
    float m = kNegInf;
    for (int64_t j = tid; j < a.V; j += kLpVjpThreads) m = fmaxf(m, Elem<T>::load(r.src + j * ES));
    m = block_max<kLpVjpThreads>(m, red[0]);
    double s, unused;
    far_sums<T, false>(r.src, a.V, m, a.c, tid, kLpVjpThreads, s, unused);
    w.hi = log2f(block_sum<kLpVjpThreads>(static_cast<float>(s), red[1]));
    w.sub = m;
    lo = 0.0f;
    __syncthreads();
    nc = r.c_hi - from;
    load(qa, c0);
  }
  const float k = ex2(-lo);
  w.a = -(gl + gH * H) * a.inv_t * k;
  w.b = -gH * kLn2 * a.inv_t * k;
  w.gt = gl * a.inv_t;
  w.x0 = (w.hi - 512.0f) / a.c;
  // (not far: |hi| < 1478, so x0's rounding to bf16 moves y by less than 8 there)
  const uint32_t low = ES == 4 ? __float_as_uint(w.x0) : pack_bf16x2(w.x0, w.x0);
  const int64_t tb = r.lead + t * ES - 16 * from;  // the given token's byte in this part
  const int64_t tc = tb >> 4;
  const int tj = static_cast<int>((tb & 15) / ES);
  auto put = [&](const uint4 (&q)[kBatch], int64_t at) {
    uint8_t* const p = gbase + 16 * (at + lane);
    const int64_t ti = tc - at - lane;  // 32 i: the token lies in this lane's chunk i
    if (!far && at + kBatchChunks <= nc) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        lp_vjp_chunk<T, false>(q[i], w, low, a.c, a.c_lo, ti == i * kSegChunks ? tj : -1, p + 16 * kSegChunks * i, congruent);
    } else {
#pragma unroll 1
      for (int i = 0; i < kBatch; ++i) {
        if (at + i * kSegChunks + lane >= nc) break;
        const uint4 qi = i == 0 ? q[0] : i == 1 ? q[1] : i == 2 ? q[2] : q[3];
        const int tji = ti == i * kSegChunks ? tj : -1;
        if (far) lp_vjp_chunk<T, true>(qi, w, low, a.c, a.c_lo, tji, p + 16 * kSegChunks * i, congruent);
        else lp_vjp_chunk<T, false>(qi, w, low, a.c, a.c_lo, tji, p + 16 * kSegChunks * i, congruent);
      }
    }
  };
  while (c0 < nc) {
    if (c0 + kStep < nc) load(qb, c0 + kStep);
    put(qa, c0);
    c0 += kStep;
    if (c0 >= nc) break;
    if (c0 + kStep < nc) load(qa, c0 + kStep);
    put(qb, c0);
    c0 += kStep;
  }
  if (e >= 0) {
    const float g = far ? vjp_element<T, true>(edge, w, a.c, a.c_lo) : vjp_element<T, false>(edge, w, a.c, a.c_lo);
    Elem<T>::store(dst + e * ES, g + (e == t ? w.gt : 0.0f));
  }
}

int token_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n > 0 ? n : 148;
}

// The lowest logit that keeps x c finite, as packed bf16 or fp32 bits.
uint32_t low_bits(float c, int es) {
  const float low = -std::min(3.3e38f, 3.3e38f / c);
  uint32_t b;
  std::memcpy(&b, &low, 4);
  return es == 4 ? b : (b >> 16) * 0x10001u;  // truncated towards 0
}

using LogprobKernel = void (*)(LogprobArgs);

template <typename T, int TOP>
LogprobKernel logprobs_kernel_for(bool split, bool short_rows) {
  if (split) return logprobs_kernel<T, TOP, true, kLpWarps>;
  return short_rows ? logprobs_kernel<T, TOP, false, 1> : logprobs_kernel<T, TOP, false, kLpWarps>;
}
template <typename T>
LogprobKernel logprobs_kernel_for(int top, bool split, bool short_rows) {
  return top == kTopNone   ? logprobs_kernel_for<T, kTopNone>(split, short_rows)
         : top == kTopWarp ? logprobs_kernel_for<T, kTopWarp>(split, short_rows)
                           : logprobs_kernel_for<T, kTopFine>(split, short_rows);
}

}  // namespace

gh_status_t logprobs_launch(const LogprobArgs& args, gh_dtype_t dtype, cudaStream_t stream) {
  LogprobArgs a = args;
  const int es = dtype == GH_F32 ? 4 : 2, epc = 16 / es, k = a.top_k;
  const int sms = token_sm_count();
  const int64_t chunks = a.V * es / 16;
  a.low = low_bits(a.c, es);
  // CTAs per row: as many as are resident together, each with at least one
  // batch a warp; for alternatives, at most kLpMaxSegs segments each.
  constexpr int kResident = kLpResident<kTopWarp, kLpWarps>;
  int S = 1;
  while (S < kMaxSlices &&
         ((a.B * S * 2 <= static_cast<int64_t>(sms) * kResident && chunks >= int64_t(2) * S * kLpWarps * kBatchChunks) ||
          (k > 0 && chunks > int64_t(S) * kLpMaxSegs * kSegChunks)))
    S *= 2;
  a.slices = S;
  a.slice_chunks = (chunks + S - 1) / S;
  if (a.B * S > INT32_MAX || (k > 0 && a.slice_chunks > int64_t(kLpMaxSegs) * kSegChunks)) return GH_ERR_UNSUPPORTED;

  // Segments: the largest kind with three per alternative (then about k of them
  // hold the alternatives and little else reaches their threshold); single logits
  // where even chunks are fewer than two per alternative.
  int top = kTopNone, smem = 0;
  if (k > 0) {
    const int64_t n = a.slice_chunks;
    a.seg_kind = n >= int64_t(3) * k * 32 ? kSegWarp : n >= int64_t(3) * k * 4 ? kSegQuad : n >= int64_t(2) * k ? kSegChunk : kSegElement;
    top = a.seg_kind == kSegWarp ? kTopWarp : kTopFine;
    const int64_t whole = (n + kBatchChunks - 1) / kBatchChunks * kBatchChunks;  // whole batches are stored
    const int64_t keys = a.seg_kind == kSegWarp   ? whole / 32
                         : a.seg_kind == kSegQuad ? whole / 4
                         : a.seg_kind == kSegChunk ? whole
                                                   : whole * epc;
    smem = static_cast<int>((keys + 127) / 128 * 128 * 4);
    if (S > 1) smem = tmax(smem, (S * k + 127) / 128 * 128 * 4 + S * k * 8);  // keys, and keys with positions
  }
  const bool short_rows = S == 1 && chunks <= kShortChunks && a.B > static_cast<int64_t>(sms) * kResident;
  const LogprobKernel kern = es == 4 ? logprobs_kernel_for<float>(top, S > 1, short_rows)
                                     : logprobs_kernel_for<uint16_t>(top, S > 1, short_rows);
  if (smem > 32 * 1024 && ensure_smem_limit(kern, kLpMaxSegs * 4) != cudaSuccess) return GH_ERR_CUDA;
  ProfileScope prof(GH_KERNEL_LOGPROBS, stream);
  note_launch();
  return launch_pdl(kern, dim3(static_cast<unsigned>(a.B * S)), dim3(32 * (short_rows ? 1 : kLpWarps)), smem, stream, S, a) == cudaSuccess
             ? GH_OK
             : GH_ERR_CUDA;
}

gh_status_t logprobs_vjp_launch(const LogprobVjpArgs& args, gh_dtype_t dtype, cudaStream_t stream) {
  LogprobVjpArgs a = args;
  const int64_t bytes = a.V * (dtype == GH_F32 ? 4 : 2);
  // parts of about kVjpPartBytes; smaller ones, down to 8 KiB, while the CTAs are fewer than are resident
  const int64_t resident = static_cast<int64_t>(token_sm_count()) * 8;
  int64_t parts = (bytes + kVjpPartBytes - 1) / kVjpPartBytes;
  while (a.B * parts < resident && bytes / (2 * parts) >= 8 * 1024) parts *= 2;
  a.parts = static_cast<int>(parts);
  a.part_chunks = (bytes / 16 + parts - 1) / parts;
  if (a.B * parts > INT32_MAX) return GH_ERR_UNSUPPORTED;
  ProfileScope prof(GH_KERNEL_LOGPROBS_VJP, stream);
  note_launch();
  const auto kern = dtype == GH_F32 ? logprobs_vjp_kernel<float> : logprobs_vjp_kernel<uint16_t>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(a.B * parts)), dim3(kLpVjpThreads), 0, stream, 1, a) == cudaSuccess
             ? GH_OK
             : GH_ERR_CUDA;
}

}  // namespace gh
