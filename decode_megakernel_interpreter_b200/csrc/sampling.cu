// Token probabilities and the verification of drafted tokens
// (include/mk_serve.h).  Both give a row of the vocabulary to a cluster of
// blocks: each block holds a slice, and the slices' maxima and sums meet in
// the blocks' shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>

#include "serve_common.h"

namespace cg = cooperative_groups;

namespace mk {
namespace {

__device__ __forceinline__ float up(float x) { return x; }
__device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float up(__half x) { return __half2float(x); }

// ---------------------------------------------------------------- token probabilities

constexpr int kProbThreads = 512;

// The factor log2(e) / T.  For T below kTinyT (`tiny`) it passes 32 bits, and is
// taken as 2^64 times a smaller one.  Where values are in registers every row has
// both multiplications (5 rows of 128256 take the same); the form for many rows,
// which they cost 2 % (512 rows 113 us, not 111), has a body for tiny T.
constexpr float kTinyT = 1e-37f;
struct PerT {
  float a, f;
  __device__ __forceinline__ PerT(float t, bool tiny)
      : a(tiny ? 0x1p64f : 1.f), f((float)(1.4426950408889634 / ((double)t * (double)a))) {}
  // x / T in powers of two
  __device__ __forceinline__ float operator()(float x) const { return x * a * f; }
};

// A block's part of a row, for the others of the cluster.
struct Part {
  float m, l;  // largest logit of the slice; sum of exp((z - m) / T)
  int first;   // where the largest is first
  int bad;     // a NaN
};

// Four consecutive logits as 32-bit values.
__device__ __forceinline__ float4 four(const float *z) {
  float4 v;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(z));
  return v;
}
template <class T>
__device__ __forceinline__ float4 four(const T *z) {  // 16-bit types
  uint2 w;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(z));
  T x[4];
  memcpy(x, &w, 8);
  return make_float4(up(x[0]), up(x[1]), up(x[2]), up(x[3]));
}

// probs = exp((z - max) / T) / sum.  A block of the row's cluster keeps its
// slice, 4 kN values a thread: first z, then exp((z - m) / T) with its own
// maximum m, which the rescaling to the row's maximum and sum turns into
// probabilities.  kN > 0: in registers, so that the row is read once, all loads
// of a thread at a time, and nothing but maxima and sums goes through shared
// memory; a vocabulary too large for that (kN = 0) is read three times.  Bound
// by memory: each logit read and each probability written once.
template <class T, int kN>
__global__ void __launch_bounds__(kProbThreads, kN <= 8 ? 2 : 1) probs_kernel(const T *logits, long long ls, const float *temperature, int ts,
                                                             float *probs, long long ps, int vocab, int per) {
  __shared__ Part part, warp_part[kProbThreads / 32];
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = min(rank * per, vocab), n = min(per, vocab - v0);
  const T *z = logits + row * ls + v0;
  float *out = probs + row * ps + v0;
  const float t = temperature ? temperature[row * ts] : 1.f;
  const bool greedy = t == 0.f;
  // Rows that start on 16 (or 8) bytes in both places go four values at a time:
  // the thread's j-th four are at 4 (512 j + tid); else at 2048 j + 512 e + tid.
  const bool vec = (reinterpret_cast<uintptr_t>(z) & (4 * sizeof(T) - 1)) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  const int turns = kN ? kN : (n + 4 * kProbThreads - 1) / (4 * kProbThreads);
  auto at = [&](int j, int e) { return j * 4 * kProbThreads + (vec ? tid * 4 + e : e * kProbThreads + tid); };
  float x[kN ? kN : 1][4];
  auto load = [&](int j, float (&y)[4]) {
    if (vec && at(j, 3) < n) {
      const float4 w = four(z + at(j, 0));
      y[0] = w.x, y[1] = w.y, y[2] = w.z, y[3] = w.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = at(j, e) < n ? up(z[at(j, e)]) : -INFINITY;
    }
  };
  // f(turn, its four values)
  auto each = [&](auto &&f) {
    if (kN) {
#pragma unroll
      for (int j = 0; j < kN; ++j) f(j, x[j]);
    } else {
      for (int j = 0; j < turns; ++j) {
        load(j, x[0]);
        f(j, x[0]);
      }
    }
  };
  if (kN) {
#pragma unroll
    for (int j = 0; j < kN; ++j) load(j, x[j]);
  }

  // ---- the slice's largest logit (greedy: and where it is first, and a NaN)
  float m = -INFINITY;
  int first = vocab, bad = !(t >= 0.f && t < INFINITY);
  each([&](int, const float (&y)[4]) { m = fmaxf(m, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]))); });
  if (greedy)
    each([&](int j, const float (&y)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (y[e] == m && at(j, e) < n) first = min(first, v0 + at(j, e));
        bad |= y[e] != y[e];
      }
    });
  auto join = [&](float y, int f) {
    if (y > m || (y == m && f < first)) {
      m = y;
      first = f;
    }
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) join(__shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, first, o));
  if (lane == 0) warp_part[warp] = Part{m, 0.f, first, 0};
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int w = 0; w < kProbThreads / 32; ++w) join(warp_part[w].m, warp_part[w].first);

  // ---- sum of exp((z - m) / T), in powers of two (32-bit: the logit's
  // difference, log2(e) / T and their product are each rounded once)
  const PerT c(greedy || bad ? 1.f : t, !greedy && t < kTinyT);
  const float base = m == -INFINITY ? 0.f : m;
  auto ex = [&](float y) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(c(y - base)));
    return r;
  };
  float l = 0.f;
  if (!greedy && !bad)
    each([&](int, float (&y)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = ex(y[e]);
      l += (y[0] + y[1]) + (y[2] + y[3]);
    });
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
  if (lane == 0) warp_part[warp].l = l;
  __syncthreads();
  if (tid == 0) {
    l = 0.f;
    for (int w = 0; w < kProbThreads / 32; ++w) l += warp_part[w].l;
    part = Part{m, l, first, bad};
  }
  cl.sync();
  if (tid < C) warp_part[tid] = *cl.map_shared_rank(&part, tid);
  cl.barrier_arrive();  // the others' parts are read
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  int best = vocab;
  bad = 0;
  for (int r = 0; r < C; ++r) {
    if (warp_part[r].m > M) {
      M = warp_part[r].m;
      best = warp_part[r].first;
    }
    bad |= warp_part[r].bad;
  }
  const float Mb = M == -INFINITY ? 0.f : M;
  auto to_row = [&](float y) { return exp2f(c(y - Mb)); };  // exp((y - M) / T), for a slice's largest logit y
  if (!greedy)
    for (int r = 0; r < C; ++r) L += warp_part[r].l * to_row(warp_part[r].m);
  // (a NaN among the logits shows in the sum)
  const bool none = bad || L != L || !(M > -INFINITY && M < INFINITY);
  const float scale = none || greedy ? 0.f : to_row(m) / L;

  // ---- probabilities
  each([&](int j, float (&y)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (greedy || none) y[e] = !none && v0 + at(j, e) == best ? 1.f : 0.f;
      else y[e] = (kN ? y[e] : ex(y[e])) * scale;
    }
    if (vec && at(j, 3) < n) {
      *reinterpret_cast<float4 *>(out + at(j, 0)) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at(j, e) < n) out[at(j, e)] = y[e];
    }
  });
  cl.barrier_wait();
}

// The same for many rows, where registers would hold too few of them at a time:
// a block takes its slice twice, first for the maximum and the sum, then for
// the probabilities.  What it read first (16384 values) stays in shared memory,
// the rest is read again, mostly out of L2.  Three blocks an SM, so that one
// reads while another writes.  512 rows of 128256 on a B200: 111 us, 4.7 TB/s
// of reads and writes, against 174 in registers; bound by the steps of a
// cluster (read, agree, write), not by DRAM: without shared memory, when DRAM
// saw 1.39 times the logits, it took the same, and clusters of 2 or 8 take 128.
constexpr int kStreamThreads = 512;
constexpr int kStreamTurns = 4;  // fours that a thread loads at a time
constexpr int kKeptTurns = 8;    // its first ones, which stay in shared memory
constexpr int kStreamSmem = kKeptTurns * kStreamThreads * 16;
template <class T, bool kTiny>
__device__ __forceinline__ void probs_stream_row(const T *logits, long long ls, const float t, float *probs, long long ps, int vocab,
                                                 int per) {
  extern __shared__ float4 kept[];  // a thread reads what it wrote itself
  __shared__ Part part, warp_part[kStreamThreads / 32];
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = min(rank * per, vocab), n = min(per, vocab - v0);
  const T *z = logits + row * ls + v0;
  float *out = probs + row * ps + v0;
  const bool greedy = t == 0.f;
  const int bad_t = !(t >= 0.f && t < INFINITY);
  const PerT c(greedy || bad_t ? 1.f : t, kTiny);
  const bool vec = (reinterpret_cast<uintptr_t>(z) & (4 * sizeof(T) - 1)) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  auto at = [&](int j, int e) { return j * 4 * kStreamThreads + (vec ? tid * 4 + e : e * kStreamThreads + tid); };
  const int turns = (n + 4 * kStreamThreads - 1) / (4 * kStreamThreads);
  auto load = [&](int j0, float (&y)[kStreamTurns][4]) {
#pragma unroll
    for (int j = 0; j < kStreamTurns; ++j)
      if (vec && at(j0 + j, 3) < n) {
        const float4 w = four(z + at(j0 + j, 0));
        y[j][0] = w.x, y[j][1] = w.y, y[j][2] = w.z, y[j][3] = w.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[j][e] = at(j0 + j, e) < n ? up(z[at(j0 + j, e)]) : -INFINITY;
      }
  };
  auto ex = [&](float y, float base) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(c(y - base)));
    return r;
  };
  float m = -INFINITY, l = 0.f, y[kStreamTurns][4];
  int first = vocab, bad = bad_t;
  for (int j0 = 0; j0 < turns; j0 += kStreamTurns) {
    load(j0, y);
    if (j0 < kKeptTurns)
#pragma unroll
      for (int j = 0; j < kStreamTurns; ++j) kept[(j0 + j) * kStreamThreads + tid] = make_float4(y[j][0], y[j][1], y[j][2], y[j][3]);
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kStreamTurns; ++j) top = fmaxf(top, fmaxf(fmaxf(y[j][0], y[j][1]), fmaxf(y[j][2], y[j][3])));
    if (greedy) {
#pragma unroll
      for (int j = 0; j < kStreamTurns; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bad |= y[j][e] != y[j][e];
          // (a thread meets its values in ascending order when they come by fours; else by turns)
          if (at(j0 + j, e) < n && (y[j][e] > m || (y[j][e] == m && v0 + at(j0 + j, e) < first))) {
            m = y[j][e];
            first = v0 + at(j0 + j, e);
          }
        }
    } else {
      if (top > m) {
        l *= m == -INFINITY ? 0.f : ex(m, top);
        m = top;
      }
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int j = 0; j < kStreamTurns; ++j) l += (ex(y[j][0], base) + ex(y[j][1], base)) + (ex(y[j][2], base) + ex(y[j][3], base));
    }
  }
  auto join = [&](float m2, float l2, int f2) {
    if (greedy) {
      if (m2 > m || (m2 == m && f2 < first)) {
        m = m2;
        first = f2;
      }
      return;
    }
    const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.f : top;
    l = l * ex(m, base) + l2 * ex(m2, base);
    m = top;
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) join(__shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, l, o), __shfl_xor_sync(~0u, first, o));
  if (lane == 0) warp_part[warp] = Part{m, l, first, 0};
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    const Part q = lane < kStreamThreads / 32 ? warp_part[lane] : Part{-INFINITY, 0.f, vocab, 0};
    m = q.m;
    l = q.l;
    first = q.first;
#pragma unroll
    for (int o = 16; o; o >>= 1) join(__shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, l, o), __shfl_xor_sync(~0u, first, o));
    if (lane == 0) part = Part{m, l, first, bad};
  }
  cl.sync();
  if (tid < C) warp_part[tid] = *cl.map_shared_rank(&part, tid);
  cl.barrier_arrive();  // the others' parts are read
  __syncthreads();
  m = -INFINITY, l = 0.f, first = vocab;
  bad = 0;
  for (int r = 0; r < C; ++r) {
    join(warp_part[r].m, warp_part[r].l, warp_part[r].first);
    bad |= warp_part[r].bad;
  }
  const bool none = bad || l != l || !(m > -INFINITY && m < INFINITY);
  const float scale = none || greedy ? 0.f : 1.f / l, base = none ? 0.f : m;
  for (int j0 = 0; j0 < turns; j0 += kStreamTurns) {
    if (j0 < kKeptTurns) {
#pragma unroll
      for (int j = 0; j < kStreamTurns; ++j) {
        const float4 w = kept[(j0 + j) * kStreamThreads + tid];
        y[j][0] = w.x, y[j][1] = w.y, y[j][2] = w.z, y[j][3] = w.w;
      }
    } else if (!greedy && !none) {
      load(j0, y);
    }
#pragma unroll
    for (int j = 0; j < kStreamTurns; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[j][e] = greedy || none ? (!none && v0 + at(j0 + j, e) == first ? 1.f : 0.f) : ex(y[j][e], base) * scale;
      if (vec && at(j0 + j, 3) < n) {
        __stcs(reinterpret_cast<float4 *>(out + at(j0 + j, 0)), make_float4(y[j][0], y[j][1], y[j][2], y[j][3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at(j0 + j, e) < n) out[at(j0 + j, e)] = y[j][e];
      }
    }
  }
  cl.barrier_wait();
}

template <class T>
__global__ void __launch_bounds__(kStreamThreads, 3) probs_stream_kernel(const T *logits, long long ls, const float *temperature, int ts,
                                                                         float *probs, long long ps, int vocab, int per) {
  const int row = blockIdx.x / cg::this_cluster().num_blocks();
  const float t = temperature ? temperature[row * ts] : 1.f;
  if (t > 0.f && t < kTinyT) probs_stream_row<T, true>(logits, ls, t, probs, ps, vocab, per);
  else probs_stream_row<T, false>(logits, ls, t, probs, ps, vocab, per);
}

// ---------------------------------------------------------------- verification

constexpr int kVerThreads = 256;
constexpr int kSeg = 512;  // values that a warp sums at a time: 16 per lane, in four runs of 128
constexpr int kVerCluster = 8;
constexpr int kMaxDrafted = 64;
constexpr int kMaxVerVocab = 104857600;  // its running sums take 200 KB of a block
static_assert((kMaxVerVocab / kSeg + kVerCluster - 1) / kVerCluster * sizeof(double) == 200 * 1024, "running sums");

struct Weights {  // the values r that the new token is drawn by
  const float *p, *q;
  int without;    // a token of weight 0 (-1: none)
  bool vec;       // both rows are 16-byte aligned
  // x, or 0 where it is not above 0 or not finite
  __device__ __forceinline__ static float pos(float x) { return x < INFINITY ? fmaxf(x, 0.f) : 0.f; }
  // 4 values from i on, i a multiple of 4 (0 from n on).  max(p - q, 0) as
  // p - min(q, p): the comparison in 32 bits, the exact difference in 64.
  __device__ __forceinline__ void four(int i, int n, double (&r)[4]) const {
    float a[4], b[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec && i + 4 <= n) {
      const float4 x = __ldg(reinterpret_cast<const float4 *>(p + i));
      a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
      if (q) {
        const float4 y = __ldg(reinterpret_cast<const float4 *>(q + i));
        b[0] = y.x, b[1] = y.y, b[2] = y.z, b[3] = y.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = i + k < n ? __ldg(p + i + k) : 0.f;
        if (q) b[k] = i + k < n ? __ldg(q + i + k) : 0.f;
      }
    }
    if (without >= i && without < i + 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k == without) a[k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = pos(a[k]);
      r[k] = q ? (double)a[k] - (double)fminf(pos(b[k]), a[k]) : (double)a[k];
    }
  }
};

__device__ __forceinline__ double scan_up(double x) {  // inclusive sums over the lanes
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ double scan_max(double x) {  // largest so far over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) x = fmax(x, __shfl_up_sync(~0u, x, o));
  return x;
}

// A cluster per sequence.  The tokens that stand follow from single values;
// the new token from one row of p (and q), whose 64-bit sums are taken per
// segment of kSeg values, over a block's segments, and over the cluster, always
// in one order: the token is then found in the block, the segment and the lane
// that the running sum passes u * sum in.  The lanes' sums add the same values
// up in different orders, so a running sum could come out below the one before
// it, or above it where nothing was added: each is therefore the largest so far,
// a segment of weight 0 keeps the last one's, and the last one is the block's
// sum for all.  The blocks' ranges then meet without gaps, and a segment that
// passes the goal holds a weight.  Bound by the memory latency of those steps: one sequence takes 12.3 us, 64 of 128256 tokens (66 MB of rows) 23.0 us
// (captured, B200; blocks of 512 threads 28.9 us, clusters of 4 32.5 us, for
// the longer slice of a block or the fewer sequences on the chip at a time).
__global__ void __launch_bounds__(kVerThreads, 4) verify_kernel(const mk_verify_args a) {
  extern __shared__ double seg[];  // sums of this block's segments, then running sums
  __shared__ double total;
  __shared__ int stop, again;
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = a.max_drafted, V = a.vocab;
  const float *target = a.target + b * a.target_batch_stride;
  const float *draft = a.draft ? a.draft + b * a.draft_batch_stride : nullptr;
  const int *tokens = a.tokens + (long long)b * T;
  int n = T > 0 && a.n_drafted ? a.n_drafted[b] : T;
  if (n < 0 || n > T) {
    if (tid == 0) report(a.status, MK_ERR_DEVICE_INPUT);
    n = min(max(n, 0), T);
  }
  const float *u = a.u + (long long)b * (T + 1);

  // ---- how many tokens stand
  if (tid == 0) stop = n;
  __syncthreads();
  if (tid < n) {
    const int x = tokens[tid];
    bool ok = (unsigned)x < (unsigned)V;
    if (ok) {
      const double px = (double)Weights::pos(target[tid * a.target_row_stride + x]);
      const double qx = draft ? (double)Weights::pos(draft[tid * a.draft_row_stride + x]) : 1.0;
      ok = (double)u[tid] * qx < px;
    } else {
      report(a.status, MK_ERR_DEVICE_INPUT);
    }
    if (!ok) atomicMin(&stop, tid);
  }
  __syncthreads();
  const int acc = stop;
  int *out = a.out_tokens + (long long)b * (T + 1);
  if (rank == 0) {
    if (tid == 0) a.n_accepted[b] = acc;
    if (tid <= T && tid != acc) out[tid] = tid < acc ? tokens[tid] : -1;
  }

  // ---- the new token
  const int n_seg = (V + kSeg - 1) / kSeg, per = (n_seg + C - 1) / C;
  const int s0 = min(rank * per, n_seg), s1 = min(s0 + per, n_seg);
  Weights w;
  w.p = target + acc * a.target_row_stride;
  w.q = acc < n && draft ? draft + acc * a.draft_row_stride : nullptr;
  w.without = acc < n && !draft ? tokens[acc] : -1;
  w.vec = ((reinterpret_cast<uintptr_t>(w.p) | reinterpret_cast<uintptr_t>(w.q)) & 15) == 0;
  double sum = 0.0, before = 0.0;  // (warp 0)
  for (int pass = 0;; ++pass) {
    for (int s = s0 + warp; s < s1; s += kVerThreads / 32) {
      double x = 0.0, r[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w.four(s * kSeg + k * 128 + lane * 4, V, r[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) x += (r[k][0] + r[k][1]) + (r[k][2] + r[k][3]);
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
      if (lane == 0) seg[s - s0] = x;
    }
    __syncthreads();
    if (warp == 0) {
      double run = 0.0;
      for (int s = 0; s < s1 - s0; s += 32) {
        const double own = s + lane < s1 - s0 ? seg[s + lane] : 0.0, up_to = run + scan_up(own);
        const double x = scan_max(own > 0.0 ? up_to : run);
        if (s + lane < s1 - s0) seg[s + lane] = x;
        run = __shfl_sync(~0u, x, 31);  // (that of the last segment, where there are fewer)
      }
      if (lane == 0) total = run;
    }
    cl.sync();
    if (warp == 0) {
      const double x = lane < C ? *cl.map_shared_rank(&total, lane) : 0.0;
      // one after the other, so that a block's end is the next one's beginning
      sum = before = 0.0;
      for (int r = 0; r < C; ++r) {
        if (r == rank) before = sum;
        sum += __shfl_sync(~0u, x, r);
      }
      if (lane == 0) again = pass == 0 && acc < n && !(sum > 0.0);
    }
    cl.barrier_arrive();  // the others' totals are read
    __syncthreads();
    if (!again) break;  // (the same in every block)
    w.q = nullptr;      // p does not exceed q anywhere: draw by p itself
    w.without = -1;
    cl.barrier_wait();
  }
  if (warp == 0) {
    if (!(sum > 0.0)) {
      if (rank == 0 && lane == 0) out[acc] = -1;
    } else {
      float uu = u[T];
      uu = uu > 0.f ? fminf(uu, 0.99999994f) : 0.f;
      const double goal = (double)uu * sum;  // < sum
      const double mine_to = seg[max(0, s1 - s0 - 1)];
      // this block's sums go from `before` to before + mine_to
      if (s1 > s0 && before <= goal && (before + mine_to > goal)) {
        int s = s1 - s0 - 1;  // the first segment that passes the goal
        for (int x = 0; x < s1 - s0; x += 32) {
          const unsigned hit = __ballot_sync(~0u, x + lane < s1 - s0 && before + seg[x + lane] > goal);
          if (hit) {
            s = x + __ffs(hit) - 1;
            break;
          }
        }
        double run = before + (s > 0 ? seg[s - 1] : 0.0), r[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w.four((s0 + s) * kSeg + k * 128 + lane * 4, V, r[k]);
        int found = -1, last = -1;  // last: the last value above 0, where rounding lets the sum stop short
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = (s0 + s) * kSeg + k * 128 + lane * 4;
          const double mine = (r[k][0] + r[k][1]) + (r[k][2] + r[k][3]), x = scan_up(mine);
          double at = run + (x - mine);
          int hit = -1, pos = -1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            at += r[k][e];
            if (r[k][e] > 0.0) pos = i + e;
            if (hit < 0 && r[k][e] > 0.0 && at > goal) hit = i + e;
          }
          const unsigned any = __ballot_sync(~0u, hit >= 0), some = __ballot_sync(~0u, pos >= 0);
          if (any && found < 0) found = __shfl_sync(~0u, hit, __ffs(any) - 1);
          if (some) last = __shfl_sync(~0u, pos, 31 - __clz(some));
          run += __shfl_sync(~0u, x, 31);
        }
        if (lane == 0) out[acc] = found >= 0 ? found : last;
      }
    }
  }
  cl.barrier_wait();
}

}  // namespace
}  // namespace mk

using namespace mk;

namespace {
template <class T>
int launch_probs(const void *logits, int64_t ls, const float *temperature, int ts, float *probs, int64_t ps, int n, int vocab,
                 cudaStream_t st) {
  // A cluster of 8 for a large vocabulary, so that few rows still use many SMs
  // and a slice fits into registers (up to 64 values a thread).  Below that one
  // block is as fast (5 rows of 8192: 6.2 us with 1 and with 8).  Once there are
  // more such blocks than two an SM (38 rows), the form for many rows, in the
  // fewest blocks whose slices are mostly kept; in us, many / registers:
  //   24000:  32 rows  8.3/6.5   40 rows 10.0/10.3  400 rows  18/58
  //   128256: 32 rows 12.4/12.3  40 rows 16.4/18.6  400 rows  91/138
  // and with 1 / 2 / 4 blocks a row, 400 rows: 16384 13.6/16.5/30.9, 24000
  // 18.3/24.6/30.8, 32003 30.8/30.5/35.8, 50257 54.9/55.2/54.0, 128256
  // 114/107/91 (150 rows of 32003: 18.5/16.4/16.5).
  const int C = vocab >= 16384 ? 8 : 1;
  const int per = ((vocab + C - 1) / C + 15) / 16 * 16;
  const int turns = (per + 4 * kProbThreads - 1) / (4 * kProbThreads);
  void (*fn)(const T *, long long, const float *, int, float *, long long, int, int) =
      turns <= 2 ? probs_kernel<T, 2> : turns <= 4 ? probs_kernel<T, 4> : turns <= 8 ? probs_kernel<T, 8> :
      turns <= 16 ? probs_kernel<T, 16> : probs_kernel<T, 0>;
  int sms = 0, rc = serve_sms(&sms);
  if (rc) return rc;
  if (vocab >= 16384 && (long long)n * C > 2 * sms) {
    const int few = vocab <= 24576 ? 1 : vocab <= 49152 ? 2 : 4, slice = ((vocab + few - 1) / few + 15) / 16 * 16;
    static std::atomic<uint64_t> allowed;
    rc = serve_allow_smem(allowed, (const void *)probs_stream_kernel<T>, kStreamSmem);
    if (rc) return rc;
    return serve_launch(probs_stream_kernel<T>, dim3((unsigned)n * few), kStreamThreads, kStreamSmem, st, false, few, (const T *)logits,
                        (long long)ls, temperature, ts, probs, (long long)ps, vocab, slice);
  }
  return serve_launch(fn, dim3((unsigned)n * C), kProbThreads, 0, st, false, C, (const T *)logits, (long long)ls,
                      temperature, ts, probs, (long long)ps, vocab, per);
}
}  // namespace

int mk::token_probs(const void *logits, int32_t dtype, int64_t logits_stride, const float *temperature, int ts,
                    float *probs, int64_t probs_stride, int32_t n, int32_t vocab, void *stream) {
  if (!logits || !probs || n < 1 || vocab < 1 || vocab >= (1 << 30) || n > (1 << 24) || logits_stride < 0 ||
      probs_stride < 0 || (n > 1 && probs_stride < vocab))
    return MK_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  switch (dtype) {
    case MK_DTYPE_F32: return launch_probs<float>(logits, logits_stride, temperature, ts, probs, probs_stride, n, vocab, st);
    case MK_DTYPE_BF16: return launch_probs<__nv_bfloat16>(logits, logits_stride, temperature, ts, probs, probs_stride, n, vocab, st);
    case MK_DTYPE_F16: return launch_probs<__half>(logits, logits_stride, temperature, ts, probs, probs_stride, n, vocab, st);
  }
  return MK_ERR_INVALID_ARG;
}

extern "C" int mk_token_probs(const void *logits, int32_t dtype, int64_t logits_stride, const float *temperature,
                              float *probs, int64_t probs_stride, int32_t n, int32_t vocab, void *stream) {
  return token_probs(logits, dtype, logits_stride, temperature, 1, probs, probs_stride, n, vocab, stream);
}

extern "C" int mk_verify(const mk_verify_args *a, void *stream) {
  if (!a || a->batch < 1 || a->batch > 65535 || a->max_drafted < 0 || a->max_drafted > kMaxDrafted || a->vocab < 1 ||
      a->vocab >= (1 << 30) || !a->target || !a->u || !a->out_tokens || !a->n_accepted || (a->max_drafted > 0 && !a->tokens) ||
      a->target_batch_stride < 0 || a->target_row_stride < 0 || a->draft_batch_stride < 0 || a->draft_row_stride < 0)
    return MK_ERR_INVALID_ARG;
  const int C = kVerCluster;
  const size_t smem = ((size_t)(a->vocab + kSeg - 1) / kSeg + C - 1) / C * sizeof(double);
  if (a->vocab > kMaxVerVocab) return MK_ERR_UNSUPPORTED_SHAPE;
  static std::atomic<uint64_t> allowed;
  int rc = smem > 40 * 1024 ? serve_allow_smem(allowed, (const void *)verify_kernel, 200 * 1024) : MK_OK;
  if (rc) return rc;
  return serve_launch(verify_kernel, dim3((unsigned)a->batch * C), kVerThreads, smem, (cudaStream_t)stream, false, C, *a);
}
