// Token probabilities and the verification of drafted tokens
// (include/mk_serve.h).  Both give a row of the vocabulary to a cluster of
// blocks: each block holds a slice, and the slices' maxima and sums meet in
// the blocks' shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "serve_common.h"

namespace cg = cooperative_groups;

namespace mk {
namespace {

__device__ __forceinline__ float up(float x) { return x; }
__device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float up(__half x) { return __half2float(x); }

// ---------------------------------------------------------------- token probabilities

constexpr int kProbThreads = 512;

// A block's part of a row, for the others of the cluster.
struct Part {
  float m, l;  // largest logit of the slice; sum of exp((z - m) / T)
  int first;   // where the largest is first
  int bad;     // a NaN
};

template <class T>
struct alignas(16) Vec16 {
  T x[16 / sizeof(T)];
};

// probs = exp((z - max) / T) / sum.  One read of the logits: a block keeps its
// slice as 32-bit values in shared memory (kept = 1), first z, then
// exp((z - m) / T) with its own maximum m, which the rescaling to the row's
// maximum and sum turns into probabilities.  Slices that do not fit are read
// again (kept = 0).  Bound by memory: n * vocab reads and writes.
template <class T>
__global__ void __launch_bounds__(kProbThreads) probs_kernel(const T *logits, long long ls, const float *temperature,
                                                             float *probs, long long ps, int vocab, int per, int kept) {
  extern __shared__ __align__(16) float e_s[];
  __shared__ Part part, warp_part[kProbThreads / 32];
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = min(rank * per, vocab), n = min(per, vocab - v0);
  const T *z = logits + row * ls + v0;
  float *out = probs + row * ps + v0;
  const float t = temperature ? temperature[row] : 1.f;
  const bool greedy = t == 0.f;
  constexpr int kV = 16 / sizeof(T);
  const bool vec = (reinterpret_cast<uintptr_t>(z) & 15) == 0;

  // ---- the slice's largest logit
  float m = -INFINITY;
  int first = vocab, bad = !(t >= 0.f && t < INFINITY);
  auto see = [&](float x, int i) {
    if (x > m) {
      m = x;
      first = v0 + i;  // a thread meets its values in ascending order
    }
    bad |= x != x;
    if (kept) e_s[i] = x;
  };
  int i0 = 0;
  if (vec) {
    i0 = n / kV * kV;
#pragma unroll 4
    for (int i = tid * kV; i < i0; i += kProbThreads * kV) {
      const Vec16<T> w = *reinterpret_cast<const Vec16<T> *>(z + i);
#pragma unroll
      for (int k = 0; k < kV; ++k) see(up(w.x[k]), i + k);
    }
  }
#pragma unroll 4
  for (int i = i0 + tid; i < n; i += kProbThreads) see(up(z[i]), i);
  auto join = [&](float x, int f) {
    if (x > m || (x == m && f < first)) {
      m = x;
      first = f;
    }
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) join(__shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, first, o));
  bad = __any_sync(~0u, bad);
  if (lane == 0) warp_part[warp] = Part{m, 0.f, first, bad};
  __syncthreads();
  for (int w = 0; w < kProbThreads / 32; ++w) {
    join(warp_part[w].m, warp_part[w].first);
    bad |= warp_part[w].bad;
  }

  // ---- sum of exp((z - m) / T), in powers of two; log2(e) / T as two
  // numbers, so that its rounding does not grow with z - m
  const double c64 = greedy || bad ? 0.0 : 1.4426950408889634 / (double)t;
  const float c_hi = (float)c64, c_lo = (float)(c64 - (double)c_hi), base = m == -INFINITY ? 0.f : m;
  auto ex = [&](float x) {
    const float d = x - base;
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaf(d, c_hi, d == -INFINITY ? 0.f : d * c_lo)));
    return y;
  };
  float l = 0.f;
  if (!greedy) {
    auto add = [&](int i) {
      const float y = ex(kept ? e_s[i] : up(z[i]));
      if (kept) e_s[i] = y;
      l += y;
    };
    for (int i = tid * kV; i < i0; i += kProbThreads * kV)
#pragma unroll
      for (int k = 0; k < kV; ++k) add(i + k);
    for (int i = i0 + tid; i < n; i += kProbThreads) add(i);
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
  }
  __syncthreads();  // warp_part is read
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
  int at = vocab;
  bad = 0;
  for (int r = 0; r < C; ++r) {
    if (warp_part[r].m > M) {
      M = warp_part[r].m;
      at = warp_part[r].first;
    }
    bad |= warp_part[r].bad;
  }
  const float Mb = M == -INFINITY ? 0.f : M;
  auto to_row = [&](float x) {  // exp((x - M) / T), for a slice's largest logit x
    const float d = x - Mb;
    return exp2f(fmaf(d, c_hi, d == -INFINITY ? 0.f : d * c_lo));
  };
  for (int r = 0; r < C; ++r) L += warp_part[r].l * to_row(warp_part[r].m);
  const bool none = bad || !(M > -INFINITY && M < INFINITY);
  const float scale = none || greedy ? 0.f : to_row(m) / L;

  // ---- probabilities
  auto p_of = [&](int i) {
    if (greedy || none) return !none && v0 + i == at ? 1.f : 0.f;
    return (kept ? e_s[i] : ex(up(z[i]))) * scale;
  };
  const bool vec_out = vec && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  if (vec_out) {
    for (int i = tid * kV; i < i0; i += kProbThreads * kV)
#pragma unroll
      for (int k = 0; k < kV; k += 4)
        *reinterpret_cast<float4 *>(out + i + k) = make_float4(p_of(i + k), p_of(i + k + 1), p_of(i + k + 2), p_of(i + k + 3));
  } else {
    for (int i = tid * kV; i < i0; i += kProbThreads * kV)
#pragma unroll
      for (int k = 0; k < kV; ++k) out[i + k] = p_of(i + k);
  }
  for (int i = i0 + tid; i < n; i += kProbThreads) out[i] = p_of(i);
  cl.barrier_wait();
}

// ---------------------------------------------------------------- verification

constexpr int kVerThreads = 512;
constexpr int kSeg = 512;  // values that a warp sums at a time: 16 per lane, in four runs of 128
constexpr int kVerCluster = 8;
constexpr int kMaxDrafted = 64;

struct Weights {  // the values r that the new token is drawn by
  const float *p, *q;
  int without;    // a token of weight 0 (-1: none)
  bool vec;       // both rows are 16-byte aligned
  __device__ __forceinline__ static double pos(float x) { return x > 0.f && x < INFINITY ? (double)x : 0.0; }
  // 4 values from i on, i a multiple of 4 (0 from n on)
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
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = i + k == without ? 0.0 : fmax(pos(a[k]) - pos(b[k]), 0.0);
  }
};

// A cluster per sequence.  The tokens that stand follow from single values;
// the new token from one row of p (and q), whose 64-bit sums are taken per
// segment of kSeg values, per block, and over the cluster, always in that
// order: the token is then found in the block, the segment and the lane that
// the running sum passes u * sum in.  Bound by the memory latency of those
// steps for few sequences, by reading the rows for many.
__global__ void __launch_bounds__(kVerThreads) verify_kernel(const mk_verify_args a) {
  extern __shared__ double seg[];  // sums of this block's segments
  __shared__ double total;
  __shared__ int stop;
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
      const double px = Weights::pos(target[tid * a.target_row_stride + x]);
      const double qx = draft ? Weights::pos(draft[tid * a.draft_row_stride + x]) : 1.0;
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
  double sum = 0.0, before = 0.0;
  for (int pass = 0; pass < 2; ++pass) {
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
    if (tid == 0) {
      double x = 0.0;
      for (int s = 0; s < s1 - s0; ++s) x += seg[s];
      total = x;
    }
    cl.sync();
    sum = before = 0.0;
    for (int r = 0; r < C; ++r) {
      if (r == rank) before = sum;
      sum += *cl.map_shared_rank(&total, r);
    }
    cl.sync();
    if (sum > 0.0 || acc == n) break;
    w.q = nullptr;  // p does not exceed q anywhere: draw by p itself
    w.without = -1;
  }
  if (!(sum > 0.0)) {
    if (rank == 0 && tid == 0) out[acc] = -1;
    return;
  }
  float uu = u[T];
  uu = uu > 0.f ? fminf(uu, 0.99999994f) : 0.f;
  const double goal = (double)uu * sum;  // < sum
  if (!(before <= goal && before + total > goal) || warp) return;
  double run = 0.0;
  int s = 0;
  for (; s < s1 - s0 - 1 && !(before + (run + seg[s]) > goal); ++s) run += seg[s];
  run += before;
  int found = -1, last = -1;  // last: the last value above 0, where rounding lets the sum stop short
  for (int k = 0; k < 4 && found < 0; ++k) {
    double r[4];
    const int i = (s0 + s) * kSeg + k * 128 + lane * 4;
    w.four(i, V, r);
    const double mine = (r[0] + r[1]) + (r[2] + r[3]);
    double x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    double at = run + (x - mine);
    int hit = -1, pos = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      at += r[e];
      if (r[e] > 0.0) pos = i + e;
      if (hit < 0 && r[e] > 0.0 && at > goal) hit = i + e;
    }
    const unsigned any = __ballot_sync(~0u, hit >= 0), some = __ballot_sync(~0u, pos >= 0);
    if (any) found = __shfl_sync(~0u, hit, __ffs(any) - 1);
    if (some) last = __shfl_sync(~0u, pos, 31 - __clz(some));
    run += __shfl_sync(~0u, x, 31);
  }
  if (lane == 0) out[acc] = found >= 0 ? found : last;
}

}  // namespace
}  // namespace mk

using namespace mk;

namespace {
template <class T>
int launch_probs(const void *logits, int64_t ls, const float *temperature, float *probs, int64_t ps, int n, int vocab,
                 cudaStream_t st) {
  const int C = vocab >= 16384 ? 8 : 1;
  int per = (vocab + C - 1) / C;
  per = (per + 15) / 16 * 16;
  const size_t bytes = (size_t)per * 4;
  const int kept = bytes <= 200 * 1024;
  const size_t smem = kept ? bytes : 0;
  int rc = serve_code(cudaFuncSetAttribute((const void *)probs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           200 * 1024));
  if (rc) return rc;
  return serve_launch(probs_kernel<T>, dim3((unsigned)n * C), kProbThreads, smem, st, false, C, (const T *)logits,
                      (long long)ls, temperature, probs, (long long)ps, vocab, per, kept);
}
}  // namespace

extern "C" int mk_token_probs(const void *logits, int32_t dtype, int64_t logits_stride, const float *temperature,
                              float *probs, int64_t probs_stride, int32_t n, int32_t vocab, void *stream) {
  if (!logits || !probs || n < 1 || vocab < 1 || vocab >= (1 << 30) || n > (1 << 24) || logits_stride < 0 ||
      probs_stride < 0 || (n > 1 && probs_stride < vocab))
    return MK_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  switch (dtype) {
    case MK_DTYPE_F32: return launch_probs<float>(logits, logits_stride, temperature, probs, probs_stride, n, vocab, st);
    case MK_DTYPE_BF16: return launch_probs<__nv_bfloat16>(logits, logits_stride, temperature, probs, probs_stride, n, vocab, st);
    case MK_DTYPE_F16: return launch_probs<__half>(logits, logits_stride, temperature, probs, probs_stride, n, vocab, st);
  }
  return MK_ERR_INVALID_ARG;
}

extern "C" int mk_verify(const mk_verify_args *a, void *stream) {
  if (!a || a->batch < 1 || a->batch > 65535 || a->max_drafted < 0 || a->max_drafted > kMaxDrafted || a->vocab < 1 ||
      a->vocab >= (1 << 30) || !a->target || !a->u || !a->out_tokens || !a->n_accepted || (a->max_drafted > 0 && !a->tokens) ||
      a->target_batch_stride < 0 || a->target_row_stride < 0 || a->draft_batch_stride < 0 || a->draft_row_stride < 0)
    return MK_ERR_INVALID_ARG;
  const int C = kVerCluster;
  const size_t smem = ((size_t)(a->vocab + kSeg - 1) / kSeg + C - 1) / C * sizeof(double);
  if (smem > 200 * 1024) return MK_ERR_UNSUPPORTED_SHAPE;
  int rc = smem > 40 * 1024 ? serve_code(cudaFuncSetAttribute((const void *)verify_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) : MK_OK;
  if (rc) return rc;
  return serve_launch(verify_kernel, dim3((unsigned)a->batch * C), kVerThreads, smem, (cudaStream_t)stream, false, C, *a);
}
