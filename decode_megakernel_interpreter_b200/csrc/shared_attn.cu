// Decode attention for a batch that shares a prefix (include/mk_serve.h).
//
// Every query row (sequence, token, head) attends over the prefix and over its
// sequence's own positions.  The rows of one K/V head that read the prefix
// form one matrix, so a prefix tile is read once and multiplied by all of
// them; the own parts are small matrices of n_tokens * group rows each.  Both
// give partial results (unnormalised o, row maximum m, row sum l), which a
// second kernel joins:
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,  M = max_s m_s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "serve_common.h"

namespace mk {
namespace {

constexpr int kRows = 16;    // query rows of an item (one m16 matrix instruction)
constexpr int kKeys = 64;    // positions of a tile
constexpr int kWarps = 4;    // each takes kKeys / kWarps positions of a tile
constexpr int kStages = 3;   // tiles in shared memory
constexpr int kMaxRowsB = 1024;

struct AttnDev {
  const char *q, *k, *v;
  char *out;
  float *lse;
  const int *prefix_pages, *prefix_len, *table, *lens;
  int32_t *status;
  long long q_bs, q_ts, q_hs, o_bs, o_ts, o_hs, kv_ps, kv_hs, kv_rs;  // bytes
  int B, T, nq, nkv, G, page, n_pages, n_prefix_pages, table_width;
  float scale2;  // |scale| * log2(e): scores in powers of two
  uint32_t flip; // sign bits of two elements of q: set for a negative scale
  int n_prefix_items, own_tiles, n_items;  // items: prefix [kv head][row tile], then own [b][kv head][row tile]
  float *part_o;    // [slot][kRows][d]
  float2 *part_ml;  // [slot][kRows]
};

// The work as a line of K/V tiles: item i owns tiles [start(i), start(i + 1));
// block c of N takes the c-th equal share of the line, so every block reads
// the same number of tiles whatever the lengths are.  A block's part of an
// item is one partial result, in slot c + i: walking along the line, each
// new part has a larger block or a larger item.
struct Line {
  int prefix, prefix_tiles;  // positions and tiles of the prefix
  long long own0, total;     // where the own items begin, and the end
  long long N;               // blocks that share it, every one with a tile at least
};

// positions of sequence b (negative: unused), cut to its pages
__device__ __forceinline__ int seq_len(const AttnDev &p, int b) {
  const int cap = p.table_width * p.page, n = p.lens[b];
  if (n > cap) report(p.status, MK_ERR_DEVICE_INPUT);
  return min(n, cap);
}
__device__ __forceinline__ int own_len(const AttnDev &p, int b, int prefix) { return max(0, seq_len(p, b) - prefix); }

// Tiles of one own item of each sequence as prefix sums: sum[b] = tiles of the
// sequences before b (sum: B + 1 ints).  Called by the whole block.
__device__ Line make_line(const AttnDev &p, int blocks, int *sum, int *red) {
  Line l;
  const long long cap = (long long)p.n_prefix_pages * p.page;
  long long n = p.n_prefix_pages > 0 ? p.prefix_len[0] : 0;
  if ((n < 0 || n > cap) && threadIdx.x == 0) report(p.status, MK_ERR_DEVICE_INPUT);
  l.prefix = (int)max(0ll, min(n, cap));
  l.prefix_tiles = (l.prefix + kKeys - 1) / kKeys;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = (p.B + blockDim.x - 1) / blockDim.x;
  const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += (own_len(p, b, l.prefix) + kKeys - 1) / kKeys;
  int x = warp_incl_sum(mine);
  if (lane == 31) red[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += red[w];
  x -= mine;
  for (int b = b0; b < b1; ++b) {
    sum[b] = x;
    x += (own_len(p, b, l.prefix) + kKeys - 1) / kKeys;
  }
  if (b0 < b1 && b1 == p.B) sum[p.B] = x;
  __syncthreads();
  l.own0 = (long long)p.n_prefix_items * l.prefix_tiles;
  l.total = l.own0 + (long long)sum[p.B] * p.nkv * p.own_tiles;
  l.N = min((long long)blocks, l.total);
  return l;
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ float exp2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <class T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ bool finite2(uint32_t w) {
    return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u;
  }
};
template <>
struct Num<__half> {
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  }
  static __device__ __forceinline__ bool finite2(uint32_t w) {
    return (w & 0x7c00u) != 0x7c00u && (w & 0x7c000000u) != 0x7c000000u;
  }
};

// Shared memory of the partial kernel: the tiles (K then V of each stage),
// reused at an item's end for the warps' partials; then the line's sums.
template <int D>
constexpr int tile_bytes() {
  return kKeys * D * 2;
}
template <int D>
constexpr int smem_tiles() {
  return kStages * 2 * tile_bytes<D>();
}

// Where 16-byte chunk c of row r of a tile stands: rows of D elements, the
// chunks of each group of eight exchanged by the row number so that eight rows'
// same chunk lies in eight different banks groups.
template <int D>
__device__ __forceinline__ uint32_t at(int r, int c) {
  return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32) part_kernel(const AttnDev p) {
  extern __shared__ __align__(128) char sm[];
  __shared__ int red[kWarps];
  __shared__ float m_s[kWarps][kRows], l_s[kWarps][kRows];
  int *sum = reinterpret_cast<int *>(sm + smem_tiles<D>());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t sm0 = smem_addr(sm);
  pdl_wait();
  pdl_trigger();
  const Line line = make_line(p, gridDim.x, sum, red);
  const long long c = blockIdx.x;
  if (c >= line.N) return;
  long long t0 = c * line.total / line.N;
  const long long t_end = (c + 1) * line.total / line.N;

  while (t0 < t_end) {
    // ---- which item, and which of its tiles
    int item, kv, row0, n_rows, lo, hi;  // rows row0.. of the item's row list; positions [lo, hi) of the sequence
    int b = -1;                          // own item's sequence
    long long item_t0, item_t1;
    if (t0 < line.own0) {
      item = (int)(t0 / line.prefix_tiles);
      item_t0 = (long long)item * line.prefix_tiles;
      item_t1 = item_t0 + line.prefix_tiles;
      const int tiles = p.n_prefix_items / p.nkv;
      kv = item / tiles;
      row0 = item % tiles * kRows;
      n_rows = min(kRows, p.B * p.T * p.G - row0);
      lo = 0;
      hi = line.prefix;
    } else {
      const int per = p.nkv * p.own_tiles;
      const int y = (int)((t0 - line.own0) / per);  // sum[b] <= y < sum[b + 1]
      int x0 = 0, x1 = p.B;
      while (x1 - x0 > 1) {
        const int mid = (x0 + x1) / 2;
        if (sum[mid] <= y) x0 = mid;
        else x1 = mid;
      }
      b = x0;
      const int nt = sum[b + 1] - sum[b];
      const long long base = line.own0 + (long long)sum[b] * per;
      const int k = (int)((t0 - base) / nt);
      item = p.n_prefix_items + b * per + k;
      item_t0 = base + (long long)k * nt;
      item_t1 = item_t0 + nt;
      kv = k / p.own_tiles;
      row0 = k % p.own_tiles * kRows;
      n_rows = min(kRows, p.T * p.G - row0);
      lo = line.prefix;
      hi = line.prefix + own_len(p, b, line.prefix);
    }
    const int first = (int)(t0 - item_t0), n_tiles = (int)(min(t_end, item_t1) - t0);
    t0 += n_tiles;

    // ---- this thread's rows: r and r + 8 of the tile (g = lane / 4)
    auto row_of = [&](int r, int &rb, int &rt, int &rh) {
      const int x = row0 + r;
      rh = kv * p.G + x % p.G;
      rt = x / p.G % p.T;
      rb = b >= 0 ? b : x / p.G / p.T;
    };
    uint32_t qf[D / 16][4];
    int sees[2], min_sees = hi;  // positions that the row sees
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane / 4 + 8 * h;
      sees[h] = 0;
      const char *qp = nullptr;
      if (r < n_rows) {
        int rb, rt, rh;
        row_of(r, rb, rt, rh);
        sees[h] = max(0, max(seq_len(p, rb), 0) - (p.T - 1 - rt));
        qp = p.q + rb * p.q_bs + rt * p.q_ts + rh * p.q_hs;
        min_sees = min(min_sees, sees[h]);
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][h] = qp ? *reinterpret_cast<const uint32_t *>(qp + (k * 16 + (lane & 3) * 2) * 2) ^ p.flip : 0u;
        qf[k][h + 2] = qp ? *reinterpret_cast<const uint32_t *>(qp + (k * 16 + 8 + (lane & 3) * 2) * 2) ^ p.flip : 0u;
      }
    }
    min_sees = __reduce_min_sync(0xffffffffu, min_sees);

    const int *list = b >= 0 ? p.table + (long long)b * p.table_width : p.prefix_pages;
    auto load_tile = [&](int i) {  // tile first + i into stage i % kStages
      const uint32_t dst = sm0 + (i % kStages) * 2 * tile_bytes<D>();
      const int pos0 = lo + (first + i) * kKeys;
      constexpr int kChunks = D / 8, kPerPass = kWarps * 32 / kChunks;  // rows of one pass of the block
#pragma unroll
      for (int x = 0; x < kKeys / kPerPass; ++x) {
        const int r = x * kPerPass + tid / kChunks, ch = tid % kChunks, pos = pos0 + r;
        const bool live = pos < hi;
        long long off = 0;
        if (live) {
          const int pi = pos / p.page;
          int pg = list[pi];
          if ((unsigned)pg >= (unsigned)p.n_pages) {
            report(p.status, MK_ERR_DEVICE_INPUT);
            pg = 0;
          }
          off = (long long)pg * p.kv_ps + kv * p.kv_hs + (pos - pi * p.page) * p.kv_rs + ch * 16;
        }
        cp16(dst + at<D>(r, ch), p.k + off, live);
        cp16(dst + tile_bytes<D>() + at<D>(r, ch), p.v + off, live);
      }
    };

    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < n_tiles) load_tile(i);
      cp_commit();
    }
    for (int i = 0; i < n_tiles; ++i) {
      cp_wait<kStages - 2>();
      __syncthreads();
      if (i + kStages - 1 < n_tiles) load_tile(i + kStages - 1);
      cp_commit();
      const uint32_t kt = sm0 + (i % kStages) * 2 * tile_bytes<D>(), vt = kt + tile_bytes<D>();
      const int key0 = warp * (kKeys / kWarps);  // this warp's 16 positions of the tile
      const int pos0 = lo + (first + i) * kKeys + key0;
      if (pos0 >= hi) continue;
      // ---- scores: 16 rows x 16 positions
      float s[2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t kf[4];  // positions 0-7 and 8-15, elements 0-7 and 8-15 of this step
        ldsm4(kf, kt + at<D>(key0 + (lane & 7) + (lane >> 4) * 8, k * 2 + ((lane >> 3) & 1)));
        Num<T>::mma(s[0], qf[k], kf[0], kf[1]);
        Num<T>::mma(s[1], qf[k], kf[2], kf[3]);
      }
      const bool edge = pos0 + 16 > min(min_sees, hi);
      if (edge) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int pos = pos0 + n * 8 + (lane & 3) * 2 + (e & 1);
            if (pos >= min(sees[e >> 1], hi)) s[n][e] = -INFINITY;
          }
      }
      // ---- running maximum and sum of each row (32-bit; scores in powers of two)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        // (a row that has seen nothing yet: x = -inf, whatever the scale)
        const float mn = fmaxf(m[h], x == -INFINITY ? x : x * p.scale2), base = mn == -INFINITY ? 0.f : mn;
        const float f = exp2_(m[h] - base);
        m[h] = mn;
        float t = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y = s[n][2 * h + e];
            s[n][2 * h + e] = y == -INFINITY ? 0.f : exp2_(fmaf(y, p.scale2, -base));
            t += s[n][2 * h + e];
          }
        l[h] = l[h] * f + t;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          o[d][2 * h] *= f;
          o[d][2 * h + 1] *= f;
        }
      }
      if (edge) {
        // A masked position's V may hold an infinity or a NaN, which p = 0
        // does not cancel in a matrix product: such a tile goes element by
        // element, without the masked positions.
        bool odd = false;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const int id = x * 32 + lane;
          const uint4 w = *reinterpret_cast<const uint4 *>(sm + (vt - sm0) + at<D>(key0 + id / (D / 8), id % (D / 8)));
          odd |= !(Num<T>::finite2(w.x) && Num<T>::finite2(w.y) && Num<T>::finite2(w.z) && Num<T>::finite2(w.w));
        }
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float w = __shfl_sync(0xffffffffu, s[j / 8][2 * h + (j & 1)], (lane & ~3) | ((j & 7) >> 1));
              if (pos0 + j >= min(sees[h], hi)) continue;
#pragma unroll
              for (int d = 0; d < D / 8; ++d) {
                const float2 v = Num<T>::unpack(
                    *reinterpret_cast<const uint32_t *>(sm + (vt - sm0) + at<D>(key0 + j, d) + (lane & 3) * 4));
                o[d][2 * h] = fmaf(w, v.x, o[d][2 * h]);
                o[d][2 * h + 1] = fmaf(w, v.y, o[d][2 * h + 1]);
              }
            }
          continue;
        }
      }
      // ---- p as two numbers of the operands' type, so that its rounding
      // (2^-9 or 2^-12 relative) does not show beside the output's own
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ph[2 * n + h] = Num<T>::pack(s[n][2 * h], s[n][2 * h + 1]);
          const float2 r = Num<T>::unpack(ph[2 * n + h]);
          pl[2 * n + h] = Num<T>::pack(s[n][2 * h] - r.x, s[n][2 * h + 1] - r.y);
        }
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t vf[4];  // positions 0-7 and 8-15 of columns 0-7, then of columns 8-15
        ldsm4t(vf, vt + at<D>(key0 + (lane & 15), d * 2 + (lane >> 4)));
        Num<T>::mma(o[2 * d], ph, vf[0], vf[1]);
        Num<T>::mma(o[2 * d], pl, vf[0], vf[1]);
        Num<T>::mma(o[2 * d + 1], ph, vf[2], vf[3]);
        Num<T>::mma(o[2 * d + 1], pl, vf[2], vf[3]);
      }
    }
    cp_wait<0>();
    __syncthreads();  // the stages become the warps' partials

    // ---- join the warps and store the block's partial of this item
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if ((lane & 3) == 0) {
        m_s[warp][lane / 4 + 8 * h] = m[h];
        l_s[warp][lane / 4 + 8 * h] = l[h];
      }
    }
    float *po = reinterpret_cast<float *>(sm);  // [warp][row][D]
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2 *>(po + (warp * kRows + lane / 4 + 8 * h) * D + d * 8 + (lane & 3) * 2) =
            make_float2(o[d][2 * h], o[d][2 * h + 1]);
    __syncthreads();
    const long long slot = c + item;
    for (int x = tid; x < n_rows * (D / 4); x += kWarps * 32) {
      const int r = x / (D / 4), d = x % (D / 4) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w][r]);
      const float base = M == -INFINITY ? 0.f : M;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_(m_s[w][r] - base);
        const float4 y = *reinterpret_cast<const float4 *>(po + (w * kRows + r) * D + d);
        a.x += f * y.x;
        a.y += f * y.y;
        a.z += f * y.z;
        a.w += f * y.w;
        L += f * l_s[w][r];
      }
      *reinterpret_cast<float4 *>(p.part_o + (slot * kRows + r) * D + d) = a;
      if (d == 0) p.part_ml[slot * kRows + r] = make_float2(M, L);
    }
    __syncthreads();  // before the next item's tiles
  }
}

// Join the partials of every row: a warp per row.
template <class T, int D>
__global__ void __launch_bounds__(128) join_kernel(const AttnDev p, int N) {
  extern __shared__ int sum[];
  __shared__ int red[4];
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const Line line = make_line(p, N, sum, red);
  const int rows = p.B * p.T * p.nq;
  for (int x = blockIdx.x * 4 + (threadIdx.x >> 5); x < rows; x += gridDim.x * 4) {
    const int h = x % p.nq, t = x / p.nq % p.T, b = x / p.nq / p.T;
    if (p.lens[b] < 0) continue;
    const int kv = h / p.G, g = h % p.G;
    float M = -INFINITY, L = 0.f, o[D / 32] = {};
    auto add = [&](int item, long long t0, long long t1, int r) {
      if (t1 <= t0) return;
      // the block that owns tile t is the largest c with c * total / N <= t;
      // with N <= total every block between the two has a part of this item
      const long long c0 = ((t0 + 1) * line.N - 1) / line.total, c1 = (t1 * line.N - 1) / line.total;
      for (long long s = c0 + item; s <= c1 + item; ++s) {
        const float2 ml = p.part_ml[s * kRows + r];
        const float mn = fmaxf(M, ml.x), base = mn == -INFINITY ? 0.f : mn;
        const float f0 = exp2_(M - base), f1 = exp2_(ml.x - base);
        M = mn;
        L = L * f0 + ml.y * f1;
        const float *a = p.part_o + (s * kRows + r) * D + lane * (D / 32);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = o[i] * f0 + a[i] * f1;
      }
    };
    const int tiles = p.n_prefix_items / p.nkv, pr = (b * p.T + t) * p.G + g;
    const int ip = kv * tiles + pr / kRows;
    add(ip, (long long)ip * line.prefix_tiles, (long long)(ip + 1) * line.prefix_tiles, pr % kRows);
    const int per = p.nkv * p.own_tiles, nt = sum[b + 1] - sum[b], w = t * p.G + g, k = kv * p.own_tiles + w / kRows;
    const long long base = line.own0 + (long long)sum[b] * per + (long long)k * nt;
    add(p.n_prefix_items + b * per + k, base, base + nt, w % kRows);
    const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;  // a NaN stays
    uint32_t *op = reinterpret_cast<uint32_t *>(p.out + b * p.o_bs + t * p.o_ts + h * p.o_hs + lane * (D / 32) * 2);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) op[i] = Num<T>::pack(L == 0.f ? 0.f : o[2 * i] * inv, L == 0.f ? 0.f : o[2 * i + 1] * inv);
    if (p.lse && lane == 0) p.lse[x] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

int check(const mk_attn_shared_args *a) {
  if (!a || a->batch < 1 || a->n_tokens < 1 || a->n_q_heads < 1 || a->n_kv_heads < 1 || a->page < 1 || a->n_pages < 1 ||
      a->n_prefix_pages < 0 || a->table_width < 1 || !std::isfinite(a->scale) || a->n_q_heads % a->n_kv_heads)
    return MK_ERR_INVALID_ARG;
  if ((a->head_dim != 64 && a->head_dim != 128) || (a->dtype != MK_DTYPE_BF16 && a->dtype != MK_DTYPE_F16) ||
      a->n_q_heads / a->n_kv_heads > 16 || a->n_tokens > 16 || (int64_t)a->batch * a->n_tokens > kMaxRowsB ||
      a->n_q_heads > 1024)
    return MK_ERR_UNSUPPORTED_SHAPE;
  // (tiles of a whole batch are counted in 32 bits)
  if ((int64_t)a->batch * ((int64_t)a->table_width * a->page / kKeys + 1) >= 1ll << 31) return MK_ERR_INVALID_ARG;
  if ((int64_t)a->table_width * a->page >= (1ll << 31) - 64 || (int64_t)a->n_prefix_pages * a->page >= (1ll << 31) - 64)
    return MK_ERR_INVALID_ARG;
  return MK_OK;
}

// Blocks of the partial kernel on this device: as many as fit at once.
constexpr int kBlocksPerSm = 2;

void fill(const mk_attn_shared_args *a, AttnDev *d) {
  d->B = a->batch;
  d->T = a->n_tokens;
  d->nq = a->n_q_heads;
  d->nkv = a->n_kv_heads;
  d->G = d->nq / d->nkv;
  d->n_prefix_items = a->n_prefix_pages > 0 ? d->nkv * ((d->B * d->T * d->G + kRows - 1) / kRows) : 0;
  d->own_tiles = (d->T * d->G + kRows - 1) / kRows;
  d->n_items = d->n_prefix_items + d->B * d->nkv * d->own_tiles;
}

int grid_of(int *out) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  *out = sms * kBlocksPerSm;
  return serve_code(e);
}

template <class T, int D>
int launch(const AttnDev &p, int N, cudaStream_t st) {
  const size_t smem = smem_tiles<D>() + sizeof(int) * (p.B + 1);
  static_assert(kStages * 2 * kKeys >= kWarps * kRows * 2, "the warps' partials fit into the tiles");
  int rc = serve_code(cudaFuncSetAttribute((const void *)part_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)smem));
  if (!rc) rc = serve_launch(part_kernel<T, D>, dim3(N), kWarps * 32, smem, st, false, 1, p);
  if (rc) return rc;
  const int rows = p.B * p.T * p.nq, grid = std::min((rows + 3) / 4, N * 4);
  return serve_launch(join_kernel<T, D>, dim3(grid), 128, sizeof(int) * (p.B + 1), st, true, 1, p, N);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int64_t mk_attn_shared_workspace_bytes(const mk_attn_shared_args *a) {
  if (check(a)) return 0;
  AttnDev d;
  fill(a, &d);
  int N = 0;
  if (grid_of(&N)) return 0;
  return ((int64_t)N + d.n_items) * kRows * (a->head_dim * 4 + 8) + 256;
}

extern "C" int mk_attn_shared(const mk_attn_shared_args *a, void *workspace, void *stream) {
  int rc = check(a);
  if (rc) return rc;
  if (!a->q || !a->k || !a->v || !a->out || !a->table || !a->lens || !workspace || !aligned_to(workspace, 256) ||
      (a->n_prefix_pages > 0 && (!a->prefix_pages || !a->prefix_len)))
    return MK_ERR_INVALID_ARG;
  const void *ptrs[] = {a->q, a->k, a->v, a->out};
  for (const void *x : ptrs)
    if (!aligned_to(x, 16)) return MK_ERR_INVALID_ARG;
  const int64_t strides[] = {a->q_batch_stride,   a->q_token_stride,  a->q_head_stride, a->out_batch_stride, a->out_token_stride,
                             a->out_head_stride,  a->page_stride,     a->kv_head_stride, a->row_stride};
  for (int64_t x : strides)
    if (x < 0 || x % 8) return MK_ERR_INVALID_ARG;
  AttnDev d = {};
  fill(a, &d);
  d.q = (const char *)a->q;
  d.k = (const char *)a->k;
  d.v = (const char *)a->v;
  d.out = (char *)a->out;
  d.lse = a->lse;
  d.prefix_pages = a->prefix_pages;
  d.prefix_len = a->prefix_len;
  d.table = a->table;
  d.lens = a->lens;
  d.status = a->status;
  d.q_bs = 2 * a->q_batch_stride;
  d.q_ts = 2 * a->q_token_stride;
  d.q_hs = 2 * a->q_head_stride;
  d.o_bs = 2 * a->out_batch_stride;
  d.o_ts = 2 * a->out_token_stride;
  d.o_hs = 2 * a->out_head_stride;
  d.kv_ps = 2 * a->page_stride;
  d.kv_hs = 2 * a->kv_head_stride;
  d.kv_rs = 2 * a->row_stride;
  d.page = a->page;
  d.n_pages = a->n_pages;
  d.n_prefix_pages = a->n_prefix_pages;
  d.table_width = a->table_width;
  d.scale2 = (float)(std::fabs((double)a->scale) * 1.4426950408889634);
  d.flip = a->scale < 0.f ? 0x80008000u : 0u;
  int N = 0;
  if ((rc = grid_of(&N))) return rc;
  const int64_t slots = (int64_t)N + d.n_items;
  d.part_o = (float *)workspace;
  d.part_ml = (float2 *)((char *)workspace + slots * kRows * a->head_dim * 4);
  cudaStream_t st = (cudaStream_t)stream;
  if (a->dtype == MK_DTYPE_BF16)
    return a->head_dim == 64 ? launch<__nv_bfloat16, 64>(d, N, st) : launch<__nv_bfloat16, 128>(d, N, st);
  return a->head_dim == 64 ? launch<__half, 64>(d, N, st) : launch<__half, 128>(d, N, st);
}
