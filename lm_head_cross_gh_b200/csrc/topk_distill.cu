// Distillation from a teacher's top logits: the row loss and the logits
// gradient from K stored entries (id, value) per row.
//
// With z = x / T, p = softmax(z) of the student's row x and q_k the teacher's
// probabilities (softmax of value / T over the row's entries, or exp(value)
// where the values are log-probabilities), Q = sum_k q_k:
//     row loss = T^2 sum_k q_k (log q_k - log p_{id_k})        (0 log 0 = 0)
//     grad_j   = scale T (Q p_j - sum_{k: id_k = j} q_k)
// (the T^2 keeps the gradient's size as T grows).  An entry whose id is -1 or
// whose value is -inf is none; a row without entries has no loss and a zero
// gradient.
//
// distill_kernel: 8 streaming warps and one for the teacher's side per row, or
// a cluster of such CTAs for long rows and small batches; three CTAs on an SM.
// The first pass sums 2^(x c - R) as the log-probabilities' forward does; the
// second reads the row again, from L2 (the rows in flight are a third of it),
// and stores the dense part scale T Q p_j; then the last warp, which has worked
// out the teacher's side and the loss meanwhile, stores the K elements that
// differ.  HBM sees one read and one write of every logit (240 MB read for 238
// MB of logits at [2368, 50257] bf16).
//
// [8192, 50257] bf16 with 32 entries: 310 to 338 us, [1024, 262144] bf16 with
// 128: 213 to 226, [4096, 50257] fp32 with 32: 313 to 326 (boards and clocks
// differ), the loss alone 161, 114 and 163.  4.4 TB/s of HBM traffic at [2368,
// 50257] bf16 with the special-function unit 62% and the issue slots 46% busy: no
// unit is full; the streaming warps wait for the row's sum between the passes
// (barrier stalls 2.4 per issue), and three CTAs on an SM do not fill that.
//
// Warps x CTAs per SM, on one board in turn, at those three shapes: 8 x 3 325 /
// 219 / 325 us, 4 x 5 351 / 242 / 356, 6 x 4 312 / 234 / 322, 7 x 3 332 / 227 / 325,
// 9 x 3 340 / 229 / 322, 12 x 2 355 / 254 / 372 (6 x 4 would need a rule on the row's
// length).  Rows are split over a cluster from 128 KiB on: at 256 KiB the rows in
// flight outgrow L2 (324 / 236 / 344), at 64 KiB the exchanges cost more (430 / 293 /
// 432).
#include "ce.h"
#include "linear_ce.h"
#include "profile.h"
#include "token_device.cuh"
#include "token_ops.h"

namespace gh {

namespace {

// Warps that stream a row (one more has the teacher's side); and for rows of up
// to 32 KiB, once there are more of them than the larger CTAs are resident
// ([3383, 5056] bf16 with 54 entries 55 -> 30 us, [4000, 16384] with 16 73 -> 66;
// 64 KiB rows lose: [4000, 32768] 108 -> 132).
constexpr int kDistillWarps = 8, kDistillShortWarps = 2;
constexpr int64_t kDistillShortChunks = 2048;
constexpr int kLaneEntries = GH_MAX_TOP_K / 32;
// CTAs of the counting kernel, its latency being a few rows' a warp ([8192, 50257]
// 332 us with 64, 323 with 256; [3383, 5056] 33.3, 30.4; [1766, 1252] 18.1, 18.4).
constexpr int kCountParts = 256;

__device__ __forceinline__ bool distill_entry(int64_t id, float v, int64_t V) {
  return id >= 0 && id < V && !(v == kNegInf);
}

// Which rows have an entry (flags, optional), and how many: each CTA writes its
// own count to parts[blockIdx.x], or adds it to *total.
__global__ void __launch_bounds__(256) distill_count_kernel(const int64_t* __restrict__ ids,
                                                            const float* __restrict__ values, int64_t B, int K,
                                                            int64_t V, int8_t* flags, unsigned int* parts,
                                                            unsigned long long* total) {
  __shared__ unsigned int n_sh;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) n_sh = 0;
  __syncthreads();
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  unsigned int n = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + warp; row < B; row += static_cast<int64_t>(gridDim.x) * 8) {
    bool any = false;
    for (int k0 = 0; k0 < K; k0 += 32) {
      const int k = k0 + lane;
      const int64_t id = k < K ? ids[row * K + k] : -1;
      const float v = k < K ? values[row * K + k] : kNegInf;
      if (id < -1 || id >= V) record_status(GH_ERR_TARGET_RANGE);
      const bool has = distill_entry(id, v, V);
      any |= __any_sync(0xffffffffu, has);
    }
    n += any ? 1 : 0;
    if (flags && lane == 0) flags[row] = any ? 1 : 0;
  }
  if (lane == 0) atomicAdd(&n_sh, n);
  __syncthreads();
  if (threadIdx.x == 0) {
    if (parts) parts[blockIdx.x] = n_sh;
    else atomicAdd(total, static_cast<unsigned long long>(n_sh));
  }
}

// Batches of up to this many rows and entries are counted by every CTA itself
// instead of by a kernel before it.  A call is the faster for that up to about 1024
// entries (11.2 us for 13.5 at [64, 1024] with 8 and [32, 1024] with 32; at 2048
// entries 11.5 for 13.5 with V = 1024, 15.0 for 13.5 with 50257); in a replayed
// graph, where a launch costs less, up to about 512 (8.0 for 9.3 us at 256, 8.7 for
// 9.3 at 512, 9.5 for 9.3 at 1024, 11.2 for 9.4 at 2048).
constexpr int kCountInside = 64;
constexpr int64_t kCountInsideEntries = 2048;

// 1 / max(n, 1) of a mean (by one warp; the same in every lane): n given, the
// sum of the counting kernel's parts, or the rows marked in has[].
__device__ __forceinline__ float distill_scale(const DistillArgs& a, const int* has, int lane) {
  if (!a.mean) return 1.0f;
  unsigned long long n = 0;
  if (a.n_valid) {
    n = *a.n_valid;
  } else if (a.parts) {
    unsigned int m = 0;
    for (int i = lane; i < a.nparts; i += 32) m += a.parts[i];
    n = __reduce_add_sync(0xffffffffu, m);
  } else {
    unsigned int m = 0;
    for (int i = lane; i < static_cast<int>(a.B); i += 32) m += has[i];
    n = __reduce_add_sync(0xffffffffu, m);
  }
  return 1.0f / static_cast<float>(n > 0 ? n : 1ull);
}

// Marks the rows of a small batch that have an entry (by a whole CTA).
__device__ __forceinline__ void mark_rows(const DistillArgs& a, int* has, int threads) {
  const int tid = static_cast<int>(threadIdx.x), B = static_cast<int>(a.B);
  for (int i = tid; i < B; i += threads) has[i] = 0;
  __syncthreads();
  for (int i = tid; i < B * a.K; i += threads) {
    const int64_t id = a.ids[i];
    if (distill_entry(id, a.values[i], a.V)) has[i / a.K] = 1;
    if (blockIdx.x == 0 && (id < -1 || id >= a.V)) record_status(GH_ERR_TARGET_RANGE);
  }
  __syncthreads();
}

// The teacher's side of a row, in shared memory (registers would be held by the
// streaming warps too).
struct Teacher {
  __align__(16) int id[GH_MAX_TOP_K];  // -1: none
  __align__(16) float q[GH_MAX_TOP_K];
  float log_q[GH_MAX_TOP_K];
  float x[GH_MAX_TOP_K];  // the student's logit at the entry
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Fills it, by one warp, lane l with entries l, l + 32, ...; returns Q.
template <typename T>
__device__ __forceinline__ float teacher_row(const DistillArgs& a, Teacher& t, int64_t row, const uint8_t* src, int lane) {
  int id[kLaneEntries];
  float log_q[kLaneEntries], q[kLaneEntries];
  float vm = kNegInf;
#pragma unroll
  for (int i = 0; i < kLaneEntries; ++i) {
    const int k = lane + 32 * i;
    id[i] = -1;
    log_q[i] = kNegInf;
    if (k < a.K) {
      const int64_t id64 = a.ids[row * a.K + k];
      const float v = a.values[row * a.K + k];
      if (distill_entry(id64, v, a.V)) {
        id[i] = static_cast<int>(id64);
        log_q[i] = v;
        vm = fmaxf(vm, v);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kLaneEntries; ++i) {
    t.id[lane + 32 * i] = id[i];
    if (id[i] >= 0) t.x[lane + 32 * i] = Elem<T>::load(src + static_cast<int64_t>(id[i]) * Elem<T>::kBytes);
  }
  float sum = 0.0f;
  if (a.renormalize) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
#pragma unroll
    for (int i = 0; i < kLaneEntries; ++i) {
      log_q[i] = id[i] >= 0 ? (log_q[i] - vm) / a.temperature : kNegInf;
      q[i] = id[i] >= 0 ? expf(log_q[i]) : 0.0f;
      sum += q[i];
    }
    sum = warp_sum(sum);
    const float log_sum = logf(sum);
#pragma unroll
    for (int i = 0; i < kLaneEntries; ++i) {
      log_q[i] -= log_sum;
      q[i] /= sum;
    }
    if (sum == sum) sum = 1.0f;  // (a NaN value makes the row NaN)
  } else {
#pragma unroll
    for (int i = 0; i < kLaneEntries; ++i) {
      q[i] = id[i] >= 0 ? expf(log_q[i]) : 0.0f;
      sum += q[i];
    }
    sum = warp_sum(sum);
  }
#pragma unroll
  for (int i = 0; i < kLaneEntries; ++i) {
    t.log_q[lane + 32 * i] = log_q[i];
    t.q[lane + 32 * i] = q[i];
  }
  __syncwarp();
  return sum;
}

// Gradient of a chunk's dense part: coef 2^y, y = (x - sub) c - r.  CONGRUENT:
// known to be at the same offset from 16 bytes as its logits.
template <typename T, bool SUB, bool CONGRUENT>
__device__ __forceinline__ void dense_chunk(const uint4& q, float sub, float c, float r, float coef, uint8_t* dst,
                                            bool congruent) {
  constexpr int ES = Elem<T>::kBytes, EPC = 16 / ES;
  float v[EPC], g[EPC];
  unpack16<T>(q, v);
  const float2 c2 = make_float2(c, c), nr = make_float2(-r, -r), k2 = make_float2(coef, coef), s2 = make_float2(-sub, -sub);
#pragma unroll
  for (int j = 0; j < EPC; j += 2) {
    float2 x = make_float2(v[j], v[j + 1]);
    if (SUB) x = __fadd2_rn(x, s2);
    const float2 y = __ffma2_rn(x, c2, nr);
    const float2 e = __fmul2_rn(make_float2(ex2(y.x), ex2(y.y)), k2);
    g[j] = e.x;
    g[j + 1] = e.y;
  }
  if (CONGRUENT || congruent) {
    __stcs(reinterpret_cast<uint4*>(dst), pack16<T>(g));
  } else {
#pragma unroll
    for (int j = 0; j < EPC; ++j) Elem<T>::store(dst + j * ES, g[j]);
  }
}

// The streaming warps' gradient stores are done (they arrive, the last warp waits).
constexpr int kStoredBarrier = 1;
template <int kThreads>
__device__ __forceinline__ void stored_arrive() {
  asm volatile("barrier.cta.arrive %0, %1;" ::"n"(kStoredBarrier), "n"(kThreads) : "memory");
}
template <int kThreads>
__device__ __forceinline__ void stored_wait() {
  asm volatile("barrier.cta.sync %0, %1;" ::"n"(kStoredBarrier), "n"(kThreads) : "memory");
}

template <int W>
struct DistillShared {
  LaneSums<W, false> sums;
  Teacher teacher;
  float4 part;  // this CTA's (maximum, reference, sum, -), read by the cluster's others
  RowDist dist;
  float coef;
  int has[kCountInside];
};

template <typename T, int W>
__global__ void __launch_bounds__(32 * (W + 1), 27 / (W + 1)) distill_kernel(DistillArgs a) {
  constexpr int kThreads = 32 * (W + 1);
  constexpr int ES = Elem<T>::kBytes;
  __shared__ DistillShared<W> sh;
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const int tid = static_cast<int>(threadIdx.x);
  pdl_wait();
  pdl_trigger();
  const int C = a.cluster;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t row = C > 1 ? blockIdx.x / C : blockIdx.x;
  const RowGeo r = row_geo<ES>(a.logits, row, a.ld, a.V);
  // this CTA's chunks of the row, and the ragged ends with the first and last
  const int64_t from = tmin(r.c_hi, r.c_lo + rank * a.slice_chunks);
  const int nc = static_cast<int>((rank == C - 1 ? r.c_hi : tmin(r.c_hi, from + a.slice_chunks)) - from);
  const uint4* const chunks = reinterpret_cast<const uint4*>(r.base) + from + lane;
  uint8_t* const dst = static_cast<uint8_t*>(a.grad) + row * a.ld_grad * ES;
  uint8_t* const gbase = dst - r.lead + 16 * from;  // this CTA's chunk i's gradient starts at gbase + 16 i
  const bool congruent = ((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(r.src)) & 15) == 0;
  constexpr int kStep = W * kBatchChunks;
  const uint32_t none = ES == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
  auto load = [&](uint4 (&q)[kBatch], int c0) {
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
  auto load_last = [&](uint4 (&q)[kBatch], int c0) {  // the second pass's: the lines may leave L2 then
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c0 + i * kSegChunks + lane < nc) q[i] = __ldcs(chunks + c0 + i * kSegChunks);
  };
  uint4 qa[kBatch], qb[kBatch];
  const int first = warp < W ? warp * kBatchChunks : nc;
  int c0 = first;
  load(qa, c0);  // before it is known whether the row counts (after it: 0.5 to 2% slower)
  if (!a.flags) mark_rows(a, sh.has, kThreads);
  const bool counts = (a.flags ? a.flags[row] : sh.has[row]) != 0;
  constexpr int kEnds = W;  // the warp of the teacher's side
  int64_t e = -1;  // a ragged-end element, in lanes of the first warp
  if (warp == 0) {
    e = edge_element(r, a.V, lane);
    if (lane < 16 ? rank != 0 : rank != C - 1) e = -1;
  }
  float edge = kNegInf;
  if (!counts) {
    if (rank == 0 && tid == 0) a.row_loss[row] = 0.0f;
    if (!a.grad) return;
    for (int c = tid; c < nc; c += kThreads) {
      if (congruent) {
        __stcs(reinterpret_cast<uint4*>(gbase + 16 * static_cast<int64_t>(c)), make_uint4(0, 0, 0, 0));
      } else {
        for (int j = 0; j < 16 / ES; ++j) Elem<T>::store(gbase + 16 * static_cast<int64_t>(c) + j * ES, 0.0f);
      }
    }
    if (e >= 0) Elem<T>::store(dst + e * ES, 0.0f);
    return;
  }

  // ---- first pass: the row's sum; the last warp has the teacher's side ----
  Teacher& t = sh.teacher;
  float ct = 1.0f, total = 0.0f;  // scale T, Q
  if (e >= 0) edge = Elem<T>::load(r.src + e * ES);
  if (warp == kEnds) {
    total = teacher_row<T>(a, t, row, r.src, lane);
    ct = distill_scale(a, sh.has, lane) * a.temperature;
  }
  WarpSums sums{kNegInf, kNegInf, {}, {}};
  float m_unused[kBatch];
  while (c0 < nc) {
    if (c0 + kStep < nc) load(qb, c0 + kStep);
    fold_batch<T, false, false>(sums, qa, a.c, 0, m_unused);
    c0 += kStep;
    if (c0 >= nc) break;
    if (c0 + kStep < nc) load(qa, c0 + kStep);
    fold_batch<T, false, false>(sums, qb, a.c, 0, m_unused);
    c0 += kStep;
  }
  // the second pass's first loads cross the exchange below
  const bool with_grad = a.grad != nullptr;
  c0 = first;
  if (with_grad) load_last(qa, c0);
  if (warp == 0) fold_lanes<false>(sums, edge, a.c);
  if (warp < W) sh.sums.post(warp, lane, sums);
  __syncthreads();
  if (warp == kEnds || C > 1) {
    SoftState st = kNoState;
    if (warp == kEnds) st = sh.sums.merge(lane);
    if (C > 1) {
      if (warp == kEnds && lane == 0) sh.part = make_float4(st.m, st.r, st.s, 0.0f);
      __syncwarp();
      cluster_arrive_release();
      cluster_wait_acquire();
      if (warp == kEnds) {
        // every CTA merges the slices in the same order
        st = kNoState;
        for (int i = 0; i < C; ++i) {
          const uint32_t p = map_to_rank(&sh.part, i);
          st = combine(st, SoftState{ld_dsmem_f32(p), ld_dsmem_f32(p + 4), ld_dsmem_f32(p + 8), 0.0f});
        }
      }
    }
    if (warp == kEnds) {
      const RowDist d = row_dist<T>(st, r.src, a.V, a.c);
      if (lane == 0) {
        sh.dist = d;
        sh.coef = d.none ? kNaN : ct * total / d.s;
      }
    }
  }
  __syncthreads();
  if (C > 1) {
    // In place, no CTA stores before every other has read what it needs of the
    // row; and none leaves before its state has been read.
    cluster_arrive_release();
    cluster_wait_acquire();
  }

  // ---- second pass: the streaming warps store the dense gradient; the last
  // warp works out the loss and the entries' elements and stores those after them ----
  const RowDist d = sh.dist;
  const float coef = sh.coef;
  if (warp == kEnds) {
    if (rank == 0) {
      float loss = 0.0f;
      for (int k = lane; k < a.K; k += 32) {
        // T (log q - log p), finite also where the entry's logit is a mask's lowest value
        const float gap = d.none ? kNaN : a.temperature * (t.log_q[k] + d.l) - (t.x[k] - d.m);
        const float q = a.temperature * t.q[k];
        if (t.id[k] >= 0 && !(q == 0.0f)) loss = fmaf(q, gap, loss);
      }
      loss = warp_sum(loss);
      if (lane == 0) a.row_loss[row] = loss;
    }
    if (!with_grad) return;
    // the gradient at the entries of this CTA's part of the row: Q p less the q
    // of every entry with that id (in place, their logits were read above)
    const int64_t lo = rank == 0 ? 0 : (16 * from - r.lead) / ES;
    const int64_t hi = rank == C - 1 ? a.V : (16 * (from + nc) - r.lead) / ES;
    int id[kLaneEntries];
    float qs[kLaneEntries];
#pragma unroll
    for (int i = 0; i < kLaneEntries; ++i) {
      id[i] = t.id[lane + 32 * i];
      qs[i] = 0.0f;
    }
    for (int j = 0; j < a.K; j += 4) {  // (-1 and 0 behind the K entries)
      const int4 other = *reinterpret_cast<const int4*>(t.id + j);
      const float4 q = *reinterpret_cast<const float4*>(t.q + j);
#pragma unroll
      for (int i = 0; i < kLaneEntries; ++i) {
        qs[i] += other.x == id[i] ? q.x : 0.0f;
        qs[i] += other.y == id[i] ? q.y : 0.0f;
        qs[i] += other.z == id[i] ? q.z : 0.0f;
        qs[i] += other.w == id[i] ? q.w : 0.0f;
      }
    }
    float fix[kLaneEntries];
#pragma unroll
    for (int i = 0; i < kLaneEntries; ++i) {
      const float p = d.none ? kNaN : ex2(fmaf(t.x[lane + 32 * i] - d.sub, a.c, -d.r)) / d.s;
      fix[i] = ct * fmaf(total, p, -qs[i]);
    }
    stored_wait<kThreads>();
#pragma unroll
    for (int i = 0; i < kLaneEntries; ++i)
      if (id[i] >= 0 && id[i] >= lo && id[i] < hi) Elem<T>::store(dst + static_cast<int64_t>(id[i]) * ES, fix[i]);
    return;
  }
  if (!with_grad) return;
  if (e >= 0) Elem<T>::store(dst + e * ES, coef * ex2(fmaf(edge - d.sub, a.c, -d.r)));
  // Full batches of ordinary rows know their alignment beforehand: 342 -> 323 us
  // at 8192 x 50257.  Two warps per CTA test it per chunk (30.4 us for 30.0 at
  // 3383 x 5056, 66.0 for 62.6 at 4000 x 16384).
  constexpr bool kKnown = W > kDistillShortWarps;
  const bool plain = d.sub == 0.0f && (!kKnown || congruent);
  auto put = [&](const uint4 (&q)[kBatch], int at) {
    uint8_t* const p = gbase + 16 * static_cast<int64_t>(at + lane);
    if (at + kBatchChunks <= nc && plain) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        dense_chunk<T, false, kKnown>(q[i], 0.0f, a.c, d.r, coef, p + 16 * kSegChunks * i, congruent);
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (at + i * kSegChunks + lane < nc)
          dense_chunk<T, true, false>(q[i], d.sub, a.c, d.r, coef, p + 16 * kSegChunks * i, congruent);
    }
  };
  while (c0 < nc) {
    if (c0 + kStep < nc) load_last(qb, c0 + kStep);
    put(qa, c0);
    c0 += kStep;
    if (c0 >= nc) break;
    if (c0 + kStep < nc) load_last(qa, c0 + kStep);
    put(qb, c0);
    c0 += kStep;
  }
  stored_arrive<kThreads>();
}

// Sum of the row losses in a fixed order, in double, and the mean's division.
__global__ void __launch_bounds__(1024) distill_reduce_kernel(DistillArgs a, float* loss) {
  __shared__ double red[32];
  __shared__ int has[kCountInside];
  pdl_wait();
  pdl_trigger();
  const int lane = static_cast<int>(threadIdx.x) & 31;
  if (a.mean && !a.n_valid && !a.parts) mark_rows(a, has, 1024);
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < a.B; i += 1024) s += static_cast<double>(a.row_loss[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    const double scale = static_cast<double>(distill_scale(a, has, lane));
    s = red[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) *loss = static_cast<float>(s * scale);
  }
}

}  // namespace

gh_status_t distill_count_launch(const int64_t* ids, const float* values, int64_t B, int K, int64_t V,
                                 unsigned long long* count, cudaStream_t stream) {
  if (cudaMemsetAsync(count, 0, sizeof(*count), stream) != cudaSuccess) return GH_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(tmin<int64_t>((B + 7) / 8, kCountParts));
  note_launch();
  return launch_pdl(distill_count_kernel, dim3(grid), dim3(256), 0, stream, 1, ids, values, B, K, V,
                    static_cast<int8_t*>(nullptr), static_cast<unsigned int*>(nullptr), count) == cudaSuccess
             ? GH_OK
             : GH_ERR_CUDA;
}

gh_status_t distill_launch(const DistillArgs& args, gh_dtype_t dtype, float* loss, cudaStream_t stream) {
  DistillArgs a = args;
  const int es = dtype == GH_F32 ? 4 : 2;
  // CTAs per row: enough that the rows in flight stay well inside L2 (a CTA's
  // part at most 128 KiB), and for small batches that the SMs have work, down
  // to 8 KiB a CTA.
  const int64_t chunks = a.V * es / 16;
  const int sms = token_sm_count();
  int C = 1;
  while (C < 8 && (chunks * 16 > C * int64_t(128 * 1024) ||
                   (a.B * C * 2 <= 2 * sms && chunks * 16 >= 2 * C * int64_t(8 * 1024))))
    C *= 2;
  a.cluster = C;
  a.slice_chunks = (chunks + C - 1) / C;
  if (a.B * C > INT32_MAX) return GH_ERR_UNSUPPORTED;  // one CTA each

  // Scratch: the counts and a flag per row (larger batches), and the row losses
  // unless the caller takes them.
  const bool inside = a.B <= kCountInside && a.B * a.K <= kCountInsideEntries;
  const size_t flag_bytes = inside ? 0 : (static_cast<size_t>(a.B) + 15) / 16 * 16 + 4 * kCountParts;
  const size_t loss_bytes = a.row_loss ? 0 : static_cast<size_t>(a.B) * sizeof(float);
  gh_status_t st = GH_OK;
  void* scratch = nullptr;
  if (flag_bytes + loss_bytes > 0) st = scratch_alloc(&scratch, flag_bytes + loss_bytes, stream);
  if (st != GH_OK) return st;
  char* p = static_cast<char*>(scratch);
  if (!a.row_loss) a.row_loss = reinterpret_cast<float*>(p + flag_bytes);
  if (!inside) {
    a.parts = reinterpret_cast<unsigned int*>(p);
    a.flags = reinterpret_cast<int8_t*>(p + 4 * kCountParts);
    a.nparts = static_cast<int>(tmin<int64_t>((a.B + 7) / 8, kCountParts));
    note_launch();
    if (launch_pdl(distill_count_kernel, dim3(static_cast<unsigned>(a.nparts)), dim3(256), 0, stream, 1, a.ids, a.values,
                   a.B, a.K, a.V, a.flags, a.parts, static_cast<unsigned long long*>(nullptr)) != cudaSuccess)
      st = GH_ERR_CUDA;
  }

  if (st == GH_OK) {
    ProfileScope prof(GH_KERNEL_DISTILL, stream);
    note_launch();
    const bool short_rows = C == 1 && chunks <= kDistillShortChunks && a.B > static_cast<int64_t>(sms) * 3;
    const int threads = 32 * ((short_rows ? kDistillShortWarps : kDistillWarps) + 1);
    const auto kern = es == 4 ? (short_rows ? distill_kernel<float, kDistillShortWarps> : distill_kernel<float, kDistillWarps>)
                              : (short_rows ? distill_kernel<uint16_t, kDistillShortWarps>
                                            : distill_kernel<uint16_t, kDistillWarps>);
    if (launch_pdl(kern, dim3(static_cast<unsigned>(a.B * C)), dim3(static_cast<unsigned>(threads)), 0, stream, C, a) != cudaSuccess)
      st = GH_ERR_CUDA;
  }
  if (st == GH_OK) {
    note_launch();
    if (launch_pdl(distill_reduce_kernel, dim3(1), dim3(1024), 0, stream, 1, a, loss) != cudaSuccess) st = GH_ERR_CUDA;
  }
  scratch_free(scratch, stream);
  return st;
}

}  // namespace gh
