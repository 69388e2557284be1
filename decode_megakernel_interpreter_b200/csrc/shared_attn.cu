// Decode attention for a batch that shares a prefix (include/mk_serve.h).
//
// Every query row (sequence, token, head) attends over the prefix and over its
// sequence's own positions.  The rows of one K/V head that read the prefix
// form one matrix, so a prefix tile is read once and multiplied by all of
// them; the own parts are small matrices of n_tokens * group rows each.  Both
// give partial results (unnormalised o, row maximum m, row sum l), which a
// last kernel joins:
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,  M = max_s m_s.
// A sequence one of whose queries ends inside the prefix does not share it:
// its whole length is then its own part, so that the shared part has no masks
// but the prefix's end.
//
// One kernel of a block per SM takes the own parts, then the prefix, and a
// second joins them.  64 sequences of 32 heads over 8 K/V heads of 128, 32768
// positions shared and up to 1024 each of their own (270 MB, 35 GF), take
// 78 us on a B200: own parts 28 us at 4.9 TB/s, prefix 36 us at 3.7 TB/s, join 7
// us.  Own parts alone reach 6.6 TB/s when they are long, the prefix of 256 rows
// 4.4 TB/s and 1110 TFLOP/s: what is lost are the starts and ends of the two
// phases.  With 7 of 8 instructions of Q K^T left out the call would gain 4 us,
// without the exponentials nothing; with the first prefix tiles brought into L2
// by the warps that are done with their own parts it took 4 us more.  Small calls are bound by the chain of dependent
// steps (lengths, line, pages, rows, partials, join): 10.3 us with hardly any
// data, 22.7 us for 16 sequences over 8192 positions of the 1B shape (25 MB).
#include <cuda.h>  // CUtensorMap (types only: the encoder is looked up at run time)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "serve_common.h"

namespace mk {
namespace {

constexpr int kRows = 16;    // query rows of an item (one m16 matrix instruction)
constexpr int kUnit = 16;    // positions that a warp takes at a time
constexpr int kWarps = 12;   // of a block; one block an SM
constexpr int kStages = 2;   // units of a warp in shared memory
// What beginning and ending an item costs a warp, in units (about 3.5 us against
// 1.9): without it the warps with many short items were the last by 15 us.
constexpr int kItemCost = 2;
// The matrix instructions cut what they add to a sum off below its last bit, so
// a long sum comes out low: by 4e-9 of itself for each position (2^18 in one sum:
// 1.2e-3, more than a step of fp16).  A part longer than this many positions is
// therefore taken in several, which are added up with the partial so far.
constexpr int kMaxSum = 16384;
constexpr int kMaxRowsB = 1024;
// A row's maximum only moves when it grows by more than 2^8: until then the
// weights are at most 2^8, which neither type nor the 32-bit sums mind, and the
// sums so far need not be rescaled.  fp16 has room above that and little below
// (what is less than 2^-25 becomes 0, which many positions of small weight would
// miss): its weights are taken in units of 2^-kShift of the maximum.
constexpr float kGrow = 8.f;

struct AttnDev {
  const char *q, *k, *v;
  char *out;
  float *lse;
  const int *prefix_pages, *prefix_len, *table, *lens;
  int32_t *status;
  long long q_bs, q_ts, q_hs, o_bs, o_ts, o_hs, kv_ps, kv_hs, kv_rs;  // bytes
  int B, T, nq, nkv, G, page, n_pages, n_prefix_pages, table_width;
  int page_shift;   // log2(page), or -1
  int page_units;   // a page is a multiple of kUnit: a unit lies in one page of a list
  float scale2;     // |scale| * log2(e): scores in powers of two
  uint32_t flip;    // sign bits of two elements of q: set for a negative scale
  int prefix_tiles;  // row tiles of a K/V head
  int n_prefix_items, own_tiles, n_items;  // items: prefix [kv head][row tile], then own [b][kv head][row tile]
  float4 *part_o;   // [slot][d / 4][kRows]
  float2 *part_ml;  // [slot][kRows]
  // for the join: how[B] (-1: unused; bit 0: shares the prefix, bit 1: has an
  // own part), then the first and last worker of each item, of this kernel and
  // of the tensor cores' (for items that have work)
  int *how;
  int2 *who, *tc_who;
  // an engine's own step (kFull): q and the output are tagged 32-bit words [batch][n_q_heads][d]
  float *tagged;
  const unsigned *epoch;
  float inv_G, inv_T;
  // the prefix on the tensor cores (tc_groups > 0; n_prefix_items is 0 then):
  // items [kv head][group of kTcGroup rows]
  int tc_groups;
  int box;         // rows of a tensor copy of K/V (0: none)
  float4 *tc_o;    // [slot][half][d / 4][kTcRows]
  float2 *tc_ml;   // [slot][half][kTcRows]
};

// `total` pieces of work shared by N workers, N <= total: worker c has
// [begin(c), begin(c + 1)), equal shares but for one piece.  The items that the
// pieces belong to follow one another along this line, so every worker does the
// same amount whatever the lengths are.  A worker's part of an item is one
// partial result, in slot c + item: walking along the line, each new part has a
// larger worker or a larger item.
struct Share {
  int total, N, each, rest;
  __device__ __forceinline__ Share(int total_, int workers) : total(total_), N(max(1, min(workers, total_))) {
    each = total / N;
    rest = total % N;
  }
  __device__ __forceinline__ int begin(int c) const { return c * each + c * rest / N; }
};

// positions of sequence b (-1: unused), cut to its pages
__device__ __forceinline__ int seq_len(const AttnDev &p, int b) {
  const int cap = p.table_width * p.page, n = p.lens[b];
  if (n > cap) report(p.status, MK_ERR_DEVICE_INPUT);
  return max(-1, min(n, cap));
}
__device__ __forceinline__ int prefix_of(const AttnDev &p) {
  const long long cap = (long long)p.n_prefix_pages * p.page, n = p.n_prefix_pages > 0 ? p.prefix_len[0] : 0;
  if ((n < 0 || n > cap) && threadIdx.x == 0) report(p.status, MK_ERR_DEVICE_INPUT);
  return (int)max(0ll, min(n, cap));
}
// How sequence b of length n goes: it shares the prefix if every query sees all
// of it; its own part begins behind it, or at 0.
__device__ __forceinline__ bool shares(const AttnDev &p, int n, int prefix) { return prefix > 0 && n - (p.T - 1) >= prefix; }
// Units of the positions [lo, hi): multiples of kUnit, the first and last may
// lie partly outside.
__device__ __forceinline__ int units(int lo, int hi) { return hi > lo ? (hi + kUnit - 1) / kUnit - lo / kUnit : 0; }
// An item's length on the line: its units, and its own cost before them.
__device__ __forceinline__ int weight(int lo, int hi) { return hi > lo ? units(lo, hi) + kItemCost : 0; }

// The line of the small items, by weight: prefix items (where the prefix does
// not go to the tensor cores), then own items; sum[b] = weights of one own item
// of each sequence before b.
struct Line {
  int prefix_weight, own0;  // own0: where the own items begin
  Share share;
  __device__ __forceinline__ Line(const AttnDev &p, int prefix, int own_weight, int workers)
      : prefix_weight(weight(0, prefix)), own0(p.n_prefix_items * prefix_weight),
        share(own0 + own_weight * p.nkv * p.own_tiles, workers) {}
};
// sum (B + 1 ints of shared memory) and the prefix's length; called by the whole block.
__device__ int make_sums(const AttnDev &p, int *sum, int *red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = (p.B + blockDim.x - 1) / blockDim.x;
  const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B), prefix = prefix_of(p);
  auto own = [&](int b) {
    const int n = seq_len(p, b);
    return weight(shares(p, n, prefix) ? prefix : 0, n);
  };
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += own(b);
  int x = warp_incl_sum(mine);
  if (lane == 31) red[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += red[w];
  x -= mine;
  for (int b = b0; b < b1; ++b) {
    sum[b] = x;
    x += own(b);
  }
  if (b0 < b1 && b1 == p.B) sum[p.B] = x;
  __syncthreads();
  if (blockIdx.x == 0)  // for the join
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
      const int n = seq_len(p, b);
      p.how[b] = n < 0 ? -1 : (shares(p, n, prefix) ? 1 : 0) | (sum[b + 1] > sum[b] ? 2 : 0);
    }
  return prefix;
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// two 32-bit numbers in a register pair
__device__ __forceinline__ unsigned long long pack2(float x, float y) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <class T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  static constexpr float kShift = 0.f;
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
  static constexpr float kShift = 7.f;  // 2^(kGrow + kShift) is below the type's largest
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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

// Add a row's partial (m, l) to the one so far; then its elements.
struct Sum {
  float now, before;  // factors
  __device__ __forceinline__ Sum(float &m, float &l, float2 so_far) {
    const float M = fmaxf(m, so_far.x), base = M == -INFINITY ? 0.f : M;
    now = exp2_(m - base);
    before = exp2_(so_far.x - base);
    m = M;
    l = l * now + so_far.y * before;
  }
  __device__ __forceinline__ float operator()(float x, float y) const { return fmaf(y, before, x * now); }
};

// Two numbers as the type's nearest, and what that leaves as another.
template <class T>
__device__ __forceinline__ void two_parts(float2 x, uint32_t &hi, uint32_t &lo) {
  hi = Num<T>::pack(x.x, x.y);
  const float2 r = Num<T>::unpack(hi);
  lo = Num<T>::pack(x.x - r.x, x.y - r.y);
}
// The values of an engine's tagged words (the two low bits are the tag).
__device__ __forceinline__ float2 untag(uint2 w) { return make_float2(__uint_as_float(w.x & ~3u), __uint_as_float(w.y & ~3u)); }

// Shared memory of the small items: each warp's stages (a unit's rows of K, then
// of V); then the line's sums.
template <int D>
constexpr int smem_stage() {
  return 2 * kUnit * D * 2;
}
template <int D>
constexpr int smem_stages() {
  return kWarps * kStages * smem_stage<D>();
}

// Where 16-byte chunk c of row r of a unit stands: rows of D elements, the
// chunks of each group of eight exchanged by the row number so that eight rows'
// same chunk lies in eight different groups of banks.
template <int D>
__device__ __forceinline__ uint32_t at(int r, int c) {
  return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

// Where a position's row is, given its page: byte offset into K or V of the
// row's head 0.
__device__ __forceinline__ int page_index(const AttnDev &p, int pos) {
  return p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page;
}
__device__ __forceinline__ long long row_offset(const AttnDev &p, int pos, int pg) {
  if ((unsigned)pg >= (unsigned)p.n_pages) {
    report(p.status, MK_ERR_DEVICE_INPUT);
    pg = 0;
  }
  return pg * p.kv_ps + (pos - page_index(p, pos) * p.page) * p.kv_rs;
}
// Copy 16 rows, the positions pos .. pos + 15, to shared memory: K and, `gap`
// bytes on, V (kBoth), or one of the two.  pg: the page of all of them (`one`),
// or of position pos + lane % 16; rows outside [lo, hi) become zeros.  to: where
// the lane's chunk of the lane's first row goes, an offset from `base` whose
// bits 4-6 are exchanged with the row number's; rows are kRow bytes apart.
template <int D, bool kBoth, int kRow>
__device__ __forceinline__ void copy_rows(const AttnDev &p, const char *k, const char *v, int kv, int pos, int lo, int hi,
                                          bool one, int pg, uint32_t base, uint32_t to, uint32_t gap) {
  const int lane = threadIdx.x & 31;
  constexpr int kChunks = D / 8, kPass = 32 / kChunks;  // rows of one instruction
  const int ch = lane % kChunks, r0 = lane / kChunks;
  const long long off = row_offset(p, pos + (one ? 0 : lane & 15), pg), head = kv * p.kv_hs + ch * 16;
  if (one && pos >= lo && pos + 16 <= hi) {
    const long long step = kPass * p.kv_rs, o = head + off + r0 * p.kv_rs;
    const char *ks = k + o, *vs = v + o;
#pragma unroll
    for (int x = 0; x < 16 / kPass; ++x, ks += step, vs += step) {
      const uint32_t dst = base + (to ^ (x * kPass & 7) << 4) + x * kPass * kRow;
      cp16(dst, ks);
      if (kBoth) cp16(dst + gap, vs);
    }
    return;
  }
#pragma unroll
  for (int x = 0; x < 16 / kPass; ++x) {
    const int r = x * kPass + r0;
    const long long o = head + (one ? off + r * p.kv_rs : __shfl_sync(0xffffffffu, off, r));
    const bool live = pos + r >= lo && pos + r < hi;
    const uint32_t dst = base + (to ^ (x * kPass & 7) << 4) + x * kPass * kRow;
    cp16(dst, k + (live ? o : 0), live);
    if (kBoth) cp16(dst + gap, v + (live ? o : 0), live);
  }
}

// A warp takes a share of the line on its own: 16 rows of Q in registers, units
// of 16 positions through two stages of shared memory, no barrier.  Such items
// are small (a sequence's own part, or a prefix with few rows), so what counts
// is how many of them wait for memory at once: 12 warps an SM, each with the
// next unit in flight.  They come before the prefix, whose partials are the
// larger ones: the join then finds those in L2.  Returns the prefix's length.
template <class T, int D, bool kFull>
__device__ __forceinline__ int small_items(const AttnDev &p, char *sm, int *red) {
  int *sum = reinterpret_cast<int *>(sm + smem_stages<D>());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kHalf = kUnit * D * 2, kStage = 2 * kHalf;
  char *const mine = sm + warp * kStages * kStage;
  const uint32_t mine_a = smem_addr(mine);
  const int prefix = make_sums(p, sum, red);
  const Line line(p, prefix, sum[p.B], gridDim.x * kWarps);
  const int c = warp * gridDim.x + blockIdx.x;  // (neighbours along the line on different SMs)
  int t0 = c < line.share.N && line.share.total > 0 ? line.share.begin(c) : 0;
  const int t_end = c < line.share.N && line.share.total > 0 ? line.share.begin(c + 1) : 0;
  int last_item = -1;

  while (t0 < t_end) {
    // ---- which item, and which of its units
    int item, kv, row0, n_rows, lo, hi;  // rows row0.. of the item's row list; positions [lo, hi) of the sequence
    int b = -1;                          // own item's sequence
    int item_t0, item_n;
    if (t0 < line.own0) {
      item = t0 / line.prefix_weight;
      item_t0 = item * line.prefix_weight;
      item_n = line.prefix_weight;
      kv = item / p.prefix_tiles;
      row0 = item % p.prefix_tiles * kRows;
      n_rows = min(kRows, p.B * p.T * p.G - row0);
      lo = 0;
      hi = prefix;
    } else {
      const int per = p.nkv * p.own_tiles, y = (t0 - line.own0) / per;  // sum[b] <= y < sum[b + 1]
      int x0 = 0, x1 = p.B;
      while (x1 - x0 > 1) {
        const int mid = (x0 + x1) / 2;
        if (sum[mid] <= y) x0 = mid;
        else x1 = mid;
      }
      b = x0;
      item_n = sum[b + 1] - sum[b];
      const int base = line.own0 + sum[b] * per, k = (t0 - base) / item_n;
      item = p.n_prefix_items + b * per + k;
      item_t0 = base + k * item_n;
      kv = k / p.own_tiles;
      row0 = k % p.own_tiles * kRows;
      n_rows = min(kRows, p.T * p.G - row0);
      hi = seq_len(p, b);
      lo = shares(p, hi, prefix) ? prefix : 0;
    }
    const int item_end = item_t0 + item_n, begin = max(t0, item_t0 + kItemCost), first = begin - item_t0 - kItemCost;
    const int n = min(min(t_end, item_end) - begin, kMaxSum / kUnit);
    t0 = n > 0 ? begin + n : min(t_end, item_end);
    if (n <= 0) continue;  // (the item's cost alone)
    const bool again = item == last_item;
    last_item = item;
    if (lane == 0) {
      if (first == 0) p.who[item].x = c;
      if (t0 == item_end) p.who[item].y = c;
    }

    const int *table = p.table + (long long)b * p.table_width;  // (not used by prefix items)
    const int key0 = (lo / kUnit + first) * kUnit;              // this part's first position
    // whether unit i is in one page: not where a sequence that does not share
    // the prefix leaves the prefix's list for its own in the middle of it
    auto one_page = [&](int i) {
      const int pos = key0 + i * kUnit;
      return p.page_units && !(lo < prefix && pos < prefix && pos + kUnit > prefix);
    };
    auto look_up = [&](int i) {  // the page of unit i, or of this lane's position of it
      const int pos = key0 + i * kUnit + (one_page(i) ? 0 : lane & 15), at = max(pos, lo);
      return i < n && at < hi ? (at < prefix ? p.prefix_pages : table)[page_index(p, at)] : 0;
    };
    auto load = [&](int i, int pg) {  // unit i into stage i % kStages
      copy_rows<D, true, D * 2>(p, p.k, p.v, kv, key0 + i * kUnit, lo, hi, one_page(i), pg, mine_a + (i & 1) * kStage,
                                at<D>(lane / (D / 8), lane % (D / 8)), kHalf);
    };
    load(0, look_up(0));
    cp_commit();
    int ahead = look_up(1);

    // ---- this thread's rows: r and r + 8 of the tile (r = lane / 4)
    uint32_t qf[D / 16][4], ql[kFull ? D / 16 : 1][4];
    int sees[2], min_sees = hi;  // positions that the row sees
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane / 4 + 8 * h, x = row0 + r;
      sees[h] = 0;
      const char *qp = nullptr;
      if (r < n_rows) {
        const int rh = kv * p.G + x % p.G, rt = x / p.G % p.T, rb = b >= 0 ? b : x / p.G / p.T;
        // (a row that does not see all of the prefix does not take this part)
        sees[h] = b < 0 ? hi : max(0, hi - (p.T - 1 - rt));
        qp = p.q + rb * p.q_bs + rt * p.q_ts + rh * p.q_hs;
        min_sees = min(min_sees, sees[h]);
      }
      if (kFull) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 y = qp ? untag(*reinterpret_cast<const uint2 *>(qp + (k * 16 + x * 8 + (lane & 3) * 2) * 4)) : make_float2(0.f, 0.f);
            two_parts<T>(y, qf[k][h + 2 * x], ql[k][h + 2 * x]);
          }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][h] = qp ? *reinterpret_cast<const uint32_t *>(qp + (k * 16 + (lane & 3) * 2) * 2) ^ p.flip : 0u;
          qf[k][h + 2] = qp ? *reinterpret_cast<const uint32_t *>(qp + (k * 16 + 8 + (lane & 3) * 2) * 2) ^ p.flip : 0u;
        }
      }
    }
    min_sees = __reduce_min_sync(0xffffffffu, min_sees);

    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int i = 0; i < n; ++i) {
      const int next = look_up(i + 2);
      cp_wait<0>();
      __syncwarp();
      if (i + 1 < n) load(i + 1, ahead);
      cp_commit();
      ahead = next;
      const int pos0 = key0 + i * kUnit;
      const char *kt = mine + (i & 1) * kStage, *vt = kt + kHalf;
      const uint32_t ka = smem_addr(kt), va = ka + kHalf;
      // ---- scores: 16 rows x 16 positions
      float s[2][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t kf[4];  // positions 0-7 and 8-15, elements 0-7 and 8-15 of this step
        ldsm4(kf, ka + at<D>((lane & 7) + (lane >> 4) * 8, k * 2 + ((lane >> 3) & 1)));
        Num<T>::mma(s[0], qf[k], kf[0], kf[1]);
        Num<T>::mma(s[1], qf[k], kf[2], kf[3]);
        if (kFull) {
          Num<T>::mma(s[0], ql[k], kf[0], kf[1]);
          Num<T>::mma(s[1], ql[k], kf[2], kf[3]);
        }
      }
      const bool edge = pos0 < lo || pos0 + kUnit > min(min_sees, hi);
      if (edge) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int pos = pos0 + n * 8 + (lane & 3) * 2 + (e & 1);
            if (pos < lo || pos >= min(sees[e >> 1], hi)) s[n][e] = -INFINITY;
          }
      }
      // ---- running maximum and sum of each row (32-bit; scores in powers of two)
      float top[2];
      bool grow = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        top[h] = x * p.scale2;
        grow |= top[h] > (m[h] == -INFINITY ? m[h] : m[h] + kGrow);
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = top[h] > m[h] ? exp2_(m[h] - top[h]) : 1.f;
          m[h] = fmaxf(m[h], top[h]);
          l[h] *= f;
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            o[d][2 * h] *= f;
            o[d][2 * h + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float base = m[h] == -INFINITY ? 0.f : m[h] - Num<T>::kShift;
        float t = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[n][2 * h + e] = exp2_(fmaf(s[n][2 * h + e], p.scale2, -base));
            t += s[n][2 * h + e];
          }
        l[h] += t;
      }
      if (edge) {
        // A masked position's V may hold an infinity or a NaN, which p = 0
        // does not cancel in a matrix product: such a tile goes element by
        // element, without the masked positions.
        bool odd = false;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const int id = x * 32 + lane;
          const uint4 w = *reinterpret_cast<const uint4 *>(vt + at<D>(id / (D / 8), id % (D / 8)));
          odd |= !(Num<T>::finite2(w.x) && Num<T>::finite2(w.y) && Num<T>::finite2(w.z) && Num<T>::finite2(w.w));
        }
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float w = __shfl_sync(0xffffffffu, s[j / 8][2 * h + (j & 1)], (lane & ~3) | ((j & 7) >> 1));
              if (pos0 + j < lo || pos0 + j >= min(sees[h], hi)) continue;
#pragma unroll
              for (int d = 0; d < D / 8; ++d) {
                const float2 v = Num<T>::unpack(
                    *reinterpret_cast<const uint32_t *>(vt + at<D>(j, d) + (lane & 3) * 4));
                o[d][2 * h] = fmaf(w, v.x, o[d][2 * h]);
                o[d][2 * h + 1] = fmaf(w, v.y, o[d][2 * h + 1]);
              }
            }
          continue;
        }
      }
      // ---- p as two numbers of the operands' type, so that its rounding
      // (2^-8 or 2^-11 relative as one) does not show beside the output's own
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          two_parts<T>(make_float2(s[n][2 * h], s[n][2 * h + 1]), ph[2 * n + h], pl[2 * n + h]);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t vf[4];  // positions 0-7 and 8-15 of columns 0-7, then of columns 8-15
        ldsm4t(vf, va + at<D>(lane & 15, d * 2 + (lane >> 4)));
        Num<T>::mma(o[2 * d], ph, vf[0], vf[1]);
        Num<T>::mma(o[2 * d + 1], ph, vf[2], vf[3]);
        Num<T>::mma(o[2 * d], pl, vf[0], vf[1]);
        Num<T>::mma(o[2 * d + 1], pl, vf[2], vf[3]);
      }
    }
    __syncwarp();  // the stages are read

    // ---- the warp's partial of this item
    const int slot = c + item;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane / 4 + 8 * h;
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      m[h] -= Num<T>::kShift;
      float2 *const ml = p.part_ml + (long long)slot * kRows + r;
      if (again) {  // (the same lanes wrote it)
        const Sum sum(m[h], l[h], r < n_rows ? *ml : make_float2(-INFINITY, 0.f));
        if (r < n_rows) {
          const float2 *from = reinterpret_cast<float2 *>(p.part_o + (long long)slot * (D / 4) * kRows + r) + (lane & 1);
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            const float2 y = from[(d * 2 + (lane >> 1 & 1)) * kRows * 2];
            o[d][2 * h] = sum(o[d][2 * h], y.x);
            o[d][2 * h + 1] = sum(o[d][2 * h + 1], y.y);
          }
        }
        __syncwarp();  // ml is read
      }
      if (r >= n_rows) continue;
      if ((lane & 3) == 0) *ml = make_float2(m[h], l[h]);
      float2 *to = reinterpret_cast<float2 *>(p.part_o + (long long)slot * (D / 4) * kRows + r) + (lane & 1);
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        to[(d * 2 + (lane >> 1 & 1)) * kRows * 2] = make_float2(o[d][2 * h], o[d][2 * h + 1]);
    }
  }
  return prefix;
}

// ---------------------------------------------------------------- the prefix on the tensor cores
//
// S = Q K^T and O += P V as matrix instructions of 128 rows (tcgen05, operands
// in shared memory, accumulators in tensor memory).  A block has two halves of
// four softmax warps, a row per thread, each half with 128 rows of a group, its
// own O, m and l, and two S of 64 positions: the tensor cores fill one while the
// softmax works on the other.  Both halves use the same K/V tiles.  (Where a
// group has 128 rows or less the second half is idle: giving it every other
// tile instead measured the same or more, up to 45.7 us against 41.0, for the
// partial results that it adds.)  K/V tiles come into a ring in the order they
// are needed, by tensor copies of the parts of a tile that lie in one page where
// pages are multiples of 16 positions, else by two warps 16 bytes a time, as is
// the prefix's last tile if it is not full (that path alone kept the tensor
// cores waiting: 42 us for 8 heads x 32768 positions x 128).  A warp for each
// half issues its matrix instructions (one warp for both spent longer on the
// waits and descriptors than the instructions took).
// P takes S's place in tensor memory, rounded to the operands' type: half a
// step (2^-8 or 2^-11) of each weight, as the output's own rounding.  With kFull
// Q and P are two numbers of the type each, the second what the first leaves,
// for an engine whose q and attention output are 32-bit numbers.

constexpr int kTcRows = 128;  // rows of a half
constexpr int kTcGroup = 2 * kTcRows;
constexpr int kTcAhead = 2;   // K tiles that are multiplied ahead of their V
constexpr int kTcKeys = 64;   // positions of a tile
// warps 0-3 and 4-7: softmax; 8 and 9: copies; 10 and 11: matrix instructions.
// (With a thirteenth warp a thread could have 128 registers only.)
constexpr int kTcThreads = kWarps * 32;
template <int D>
constexpr int tc_tile() {
  return kTcKeys * D * 2;
}
template <int D>
constexpr int tc_q() {  // a half's rows of Q
  return kTcRows * D * 2;
}
template <int D, bool kFull>
constexpr int tc_ring() {
  return D == 64 ? 16 : kFull ? 6 : 10;  // tiles of K or V in flight or in use
}
template <int D, bool kFull>
constexpr int tc_smem() {
  return (kFull ? 4 : 2) * tc_q<D>() + tc_ring<D, kFull>() * tc_tile<D>() + 1024;
}

// Byte of element chunk c (8 elements) of row r in a tile of `rows` rows: 64
// elements (128 bytes) of every row, then the next 64; the eight chunks of 128
// bytes exchanged by the row number (the 128-byte swizzle of the operand
// descriptors).
__device__ __forceinline__ uint32_t tc_at(int rows, int r, int c) {
  return (uint32_t)((c >> 3) * (rows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Operand descriptor: 128-byte swizzle, 8-row groups 1024 bytes apart.  Its low
// word is the address and lbo (from 64 elements of the leading dimension to the
// next 64; read for V only), in units of 16 bytes; the high word is the same
// for all, so that a step through a tile is one addition.
__device__ __forceinline__ uint32_t tc_low(uint32_t addr, uint32_t lbo) { return (addr >> 4) | (lbo >> 4) << 16; }
__device__ __forceinline__ uint64_t tc_desc(uint32_t low) {
  constexpr uint32_t high = (1024u >> 4) | (1u << 14) | (2u << 29);
  return (uint64_t)high << 32 | low;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t a, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_smem_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(b)), "r"(parity)
      : "memory");
  return ok != 0;
}

struct TcShared {
  uint64_t full[16], empty[16];  // ring entries
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2], drain[2];  // [half][which S]; o_full: a P V is complete
  uint32_t tmem;
  int sent[2];        // tiles that each copying warp has arrived for
  volatile int dead;  // a wait gave up
};

// Wait for a phase; false when it does not come within a second (or another
// wait has given up): every role then runs to the kernel's end.
__device__ __noinline__ bool bar_wait_long(TcShared *sh, uint64_t *b, uint32_t parity, int32_t *status) {
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  while (!bar_try(b, parity)) {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (sh->dead || t - t0 > 1000000000ull) {
      sh->dead = 1;
      report(status, MK_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool bar_wait(TcShared *sh, uint64_t *b, uint32_t parity, int32_t *status) {
  return bar_try(b, parity) || bar_wait_long(sh, b, parity, status);
}
// the same by a whole warp
__device__ __forceinline__ bool bar_wait_all(TcShared *sh, uint64_t *b, uint32_t parity, int32_t *status) {
  return __all_sync(0xffffffffu, bar_wait(sh, b, parity, status));
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(b)), "r"(bytes) : "memory");
}
// Wait for a phase until the clock says `end`.
__device__ __forceinline__ void bar_wait_until(uint64_t *b, uint32_t parity, uint64_t end) {
  uint64_t t = 0;
  while (!bar_try(b, parity) && t < end) asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
}
// A box of K or V: 64 elements from x on, of the map's number of rows.
__device__ __forceinline__ void tensor_copy(const CUtensorMap *map, uint32_t dst, int x, int row, int kv, int page, uint64_t *b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(row), "r"(kv), "r"(page), "r"(smem_addr(b))
      : "memory");
}
// Arrive on b when this thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t *b) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(b)) : "memory");
}

// The order in which the n tiles of an item pass through the ring: K of the
// first kTcAhead, then V j and K j + kTcAhead in turn, then the other V.
struct TcOrder {
  int n, ahead;
  __device__ __forceinline__ explicit TcOrder(int n_) : n(n_), ahead(min(kTcAhead, n_)) {}
  __device__ __forceinline__ int k_at(int j) const { return j < ahead ? j : 2 * j - ahead + 1; }
  __device__ __forceinline__ int v_at(int j) const { return j < n - ahead ? ahead + 2 * j : n + j; }
};

// The blocks' line of tiles.
// (An item's beginning and end cost a block as much as about 6 tiles: with that
// counted, the blocks that take parts of two items end with the others.  256
// rows of 8 K/V heads of 128 over 16384 positions: 44.4 us, with 4 counted 45.8.)
constexpr int kTcItemCost = 6;
struct TcLine {
  int tiles;
  Share share;
  __device__ __forceinline__ TcLine(const AttnDev &p, int prefix, int blocks)
      : tiles((prefix + kTcKeys - 1) / kTcKeys), share(tiles > 0 ? (tiles + kTcItemCost) * p.nkv * p.tc_groups : 0, blocks) {}
  // The next part of a block's share [t0, t_end), with kLong kMaxSum positions at most: false when there is none.
  template <bool kLong>
  __device__ __forceinline__ bool next(int &t0, int t_end, int &item, int &first, int &n) const {
    while (t0 < t_end) {
      item = t0 / (tiles + kTcItemCost);
      const int at = item * (tiles + kTcItemCost), end = min(t_end, at + tiles + kTcItemCost), from = max(t0, at + kTcItemCost);
      first = from - at - kTcItemCost;
      n = kLong ? min(end - from, kMaxSum / kTcKeys) : end - from;
      t0 = n > 0 ? from + n : end;
      if (n > 0) return true;
    }
    return false;
  }
};

// kLong: a block's share of the prefix may be longer than kMaxSum.
template <class T, int D, bool kFull, bool kLong>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_kernel(const AttnDev p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ char sm_raw[];
  __shared__ TcShared sh;
  constexpr int kRing = tc_ring<D, kFull>();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int red[kWarps];
  const uint32_t base = (smem_addr(sm_raw) + 1023) & ~1023u;
  char *sm = sm_raw + (base - smem_addr(sm_raw));
  const uint32_t ring = base + (kFull ? 4 : 2) * tc_q<D>();  // Q of both halves, then what it leaves
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      bar_init(&sh.full[i], 64);
      bar_init(&sh.empty[i], 2);  // both halves use every entry
    }
    for (int w = 0; w < 2; ++w) {
      bar_init(&sh.q_full[w], 4);
      for (int i = 0; i < 2; ++i) {
        bar_init(&sh.s_full[w][i], 1);
        bar_init(&sh.p_full[w][i], 4);
      }
      bar_init(&sh.o_full[w], 1);
    }
    bar_init(&sh.drain[0], 1);
    bar_init(&sh.drain[1], 1);
    sh.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 10)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
  pdl_wait();
  pdl_trigger();
  const int prefix = small_items<T, D, kFull>(p, sm, red), c = blockIdx.x;
  cp_wait<0>();
  fence_smem_async();  // the tensor copies reuse the small items' stages
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = sh.tmem;
  const TcLine line(p, p.tc_groups ? prefix : 0, gridDim.x);
  const int R = p.B * p.T * p.G;
  const bool any = c < line.share.N && line.tiles > 0;
  const int t_begin = any ? line.share.begin(c) : 0, t_end = any ? line.share.begin(c + 1) : 0;
  auto s_of = [&](int w, int i) { return tm + w * 128 + i * 64; };
  auto o_of = [&](int w) { return tm + 256 + w * D; };

  if (warp >= 8 && warp < 10) {
    // ---------------- copies: warp w of the two takes rows 32 w .. 32 w + 31
    // of every tile, 16 at a time
    int slot = 0, sent = 0;  // of the ring; tiles so far
    uint32_t phase = 1;   // of its `empty`: every slot is free at first
    bool ok = true;
    const int row = (warp - 8) * 32, ch = lane % (D / 8), r0 = lane / (D / 8);
    // Tensor copies take the box rows of a page at a time, 1, 2 or 4 to a tile.
    // Lane i knows the page of the i-th of the next 32 (of K, and of V).
    const int shift = p.box == 64 ? 0 : p.box == 32 ? 1 : 2, boxes = 1 << shift, tiles_mask = (32 >> shift) - 1;
    const int box_row = (lane & (boxes - 1)) * p.box;
    const uint32_t box_at = box_row * 128;
    auto step = [&]() {
      ++sent;
      if (++slot == kRing) {
        slot = 0;
        phase ^= 1;
      }
    };
    for (int t0 = t_begin, item, first, n; ok && line.next<kLong>(t0, t_end, item, first, n);) {
      const int kv = item / p.tc_groups;
      const int ahead = min(kTcAhead, n);
      int k_next = 0, v_next = 0, k_pages = 0, v_pages = 0;
      while (v_next < n) {  // (the order of TcOrder)
        const bool is_v = k_next == n || k_next - v_next >= ahead;
        const int j = is_v ? v_next++ : k_next++;
        const int pos0 = (first + j) * kTcKeys;
        const uint32_t dst = ring + slot * tc_tile<D>();
        uint64_t *full = &sh.full[slot];
        if (p.box && pos0 + kTcKeys <= prefix) {
          int pages = is_v ? v_pages : k_pages;
          if ((j & tiles_mask) == 0) {
            const unsigned pos = (unsigned)pos0 + lane * p.box;  // (up to 31 boxes past a prefix that ends just below 2^31)
            pages = pos < (unsigned)prefix ? p.prefix_pages[page_index(p, (int)pos)] : 0;
            if (is_v) v_pages = pages;
            else k_pages = pages;
          }
          int pg = __shfl_sync(0xffffffffu, pages, (j & tiles_mask) << shift | (lane & (boxes - 1)));
          ok = bar_wait_all(&sh, &sh.empty[slot], phase, p.status);
          if (!ok) break;
          if (warp == 8 && lane == 0) bar_expect(full, tc_tile<D>());
          else bar_arrive(full);
          __syncwarp();
          if (warp == 8 && lane < boxes) {
            if ((unsigned)pg >= (unsigned)p.n_pages) {
              report(p.status, MK_ERR_DEVICE_INPUT);
              pg = 0;
            }
            const int pos = pos0 + box_row, in = pos - page_index(p, pos) * p.page;
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              tensor_copy(is_v ? &v_map : &k_map, dst + x * (kTcKeys * 128) + box_at, x * 64, in, kv, pg, full);
          }
          step();
          continue;
        }
        ok = bar_wait_all(&sh, &sh.empty[slot], phase, p.status);
        if (!ok) break;
        const char *src = is_v ? p.v : p.k;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int pos = pos0 + row + x * 16, at = pos + (p.page_units ? 0 : lane & 15);
          copy_rows<D, false, 128>(p, src, src, kv, pos, 0, prefix, p.page_units, at < prefix ? p.prefix_pages[page_index(p, at)] : 0,
                                   dst, tc_at(kTcKeys, row + x * 16 + r0, ch), 0);
        }
        cp_arrive(full);
        step();
      }
    }
    cp_commit();
    cp_wait<0>();
    if (lane == 0) sh.sent[warp - 8] = sent;
  } else if (warp >= 10) {
    // ---------------- matrix instructions of half w: the warp walks as one, an
    // elected lane issues
    constexpr uint32_t kType = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    // 32-bit accumulators, both operands of this type, 128 rows; N = 64 positions, or N = D with V's
    // leading dimension the other way round
    constexpr uint32_t kS = (1u << 4) | (kType << 7) | (kType << 10) | ((kTcKeys / 8u) << 17) | ((128u / 16) << 24);
    constexpr uint32_t kO = (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) | ((uint32_t)(D / 8) << 17) | ((128u / 16) << 24);
    const int w = warp - 10;
    const uint32_t q_low = tc_low(base, 16) + w * (tc_q<D>() >> 4);
    const uint32_t k_low = tc_low(ring, 16), v_low = tc_low(ring, kTcKeys * 128);
    int g = 0;                          // ring entries before this item
    uint32_t q_phase = 0, p_phase = 0;  // one bit; bit i
    bool ok = true;
    auto take = [&](int e) {  // entry e's tile has landed
      const int x = (g + e) % kRing;
      ok = ok && bar_wait_all(&sh, &sh.full[x], ((g + e) / kRing) & 1, p.status);
      fence_smem_async();  // the copies' writes, before the tensor cores' reads
      return x;
    };
    auto scores = [&](int i, int x) {
      const uint32_t k = k_low + x * (tc_tile<D>() >> 4);
      if (elect_one()) {
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
          mma_ss(s_of(w, i), tc_desc(q_low + (e / 4 * (kTcRows * 128) + e % 4 * 32 >> 4)),
                 tc_desc(k + (e / 4 * (kTcKeys * 128) + e % 4 * 32 >> 4)), kS, e > 0);
        if (kFull)
#pragma unroll
          for (int e = 0; e < D / 16; ++e)
            mma_ss(s_of(w, i), tc_desc(q_low + (2 * tc_q<D>() + e / 4 * (kTcRows * 128) + e % 4 * 32 >> 4)),
                   tc_desc(k + (e / 4 * (kTcKeys * 128) + e % 4 * 32 >> 4)), kS, true);
        mma_commit(&sh.s_full[w][i]);
        mma_commit(&sh.empty[x]);
      }
      __syncwarp();
    };
    for (int t0 = t_begin, item, first, n; ok && line.next<kLong>(t0, t_end, item, first, n);) {
      if (w == 0 && lane == 0) {
        if (first == 0) p.tc_who[item].x = c;
        if (first + n == line.tiles) p.tc_who[item].y = c;
      }
      const TcOrder order(n);
      if (item % p.tc_groups * kTcGroup + w * kTcRows < R) {
        ok = ok && bar_wait_all(&sh, &sh.q_full[w], q_phase, p.status);
        q_phase ^= 1;
        for (int j = 0; ok && j < order.ahead; ++j) {  // tile j's S is in buffer j & 1
          const int x = take(order.k_at(j));
          if (ok) scores(j, x);
        }
        for (int j = 0, i = 0; ok && j < n; ++j, i ^= 1) {
          const int v = take(order.v_at(j));
          ok = ok && bar_wait_all(&sh, &sh.p_full[w][i], p_phase >> i & 1, p.status);  // P is in S's place
          p_phase ^= 1u << i;
          if (!ok) break;
          tc_after();
          const uint32_t low = v_low + v * (tc_tile<D>() >> 4);
          if (elect_one()) {
#pragma unroll
            for (int e = 0; e < kTcKeys / 16; ++e)
              mma_ts(o_of(w), s_of(w, i) + e * 8, tc_desc(low + e * (2048 >> 4)), kO, j > 0 || e > 0);
            if (kFull)
#pragma unroll
              for (int e = 0; e < kTcKeys / 16; ++e)
                mma_ts(o_of(w), s_of(w, i) + 32 + e * 8, tc_desc(low + e * (2048 >> 4)), kO, true);
            mma_commit(&sh.o_full[w]);
            mma_commit(&sh.empty[v]);
          }
          __syncwarp();
          if (j + kTcAhead < n) {
            const int x = take(order.k_at(j + kTcAhead));
            if (ok) scores(i, x);
          }
        }
      } else {  // no rows: the tiles only pass
        for (int e = 0; ok && e < 2 * n; ++e) {
          const int x = take(e);
          if (ok && lane == 0) bar_arrive(&sh.empty[x]);
        }
      }
      g += 2 * n;
    }
  } else if (warp < 8) {
    // ---------------- softmax: row r of half w
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    uint32_t s_phase = 0;  // bit i
    int done = 0;          // tiles of this half so far
    int last_item = -1;
    bool ok = true;
    for (int t0 = t_begin, item, first, n; ok && line.next<kLong>(t0, t_end, item, first, n);) {
      const int kv = item / p.tc_groups;
      const int row = item % p.tc_groups * kTcGroup + w * kTcRows + r;
      const bool live = row < R, any_live = row - lane < R, half_live = row - r < R;
      if (half_live) {
        // this row of Q (the S of the last item is done with the old one)
        const char *qp = nullptr;
        if (live) {
          const int rh = kv * p.G + row % p.G, rt = row / p.G % p.T, rb = row / p.G / p.T;
          qp = p.q + rb * p.q_bs + rt * p.q_ts + rh * p.q_hs;
        }
        char *const q_to = sm + w * tc_q<D>();
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          uint4 x = make_uint4(0, 0, 0, 0), rest = x;
          if (live && kFull) {
            const uint4 *f = reinterpret_cast<const uint4 *>(qp + i * 32);
            const uint4 f0 = f[0], f1 = f[1];
            two_parts<T>(untag(make_uint2(f0.x, f0.y)), x.x, rest.x);
            two_parts<T>(untag(make_uint2(f0.z, f0.w)), x.y, rest.y);
            two_parts<T>(untag(make_uint2(f1.x, f1.y)), x.z, rest.z);
            two_parts<T>(untag(make_uint2(f1.z, f1.w)), x.w, rest.w);
          } else if (live) {
            x = *reinterpret_cast<const uint4 *>(qp + i * 16);
            x.x ^= p.flip;
            x.y ^= p.flip;
            x.z ^= p.flip;
            x.w ^= p.flip;
          }
          *reinterpret_cast<uint4 *>(q_to + tc_at(kTcRows, r, i)) = x;
          if (kFull) *reinterpret_cast<uint4 *>(q_to + 2 * tc_q<D>() + tc_at(kTcRows, r, i)) = rest;
        }
        fence_smem_async();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.q_full[w]);
      }
      float m = -INFINITY, l = 0.f;
      int i = 0;  // which S
      for (int j = 0; half_live && j < n; ++j, i ^= 1) {
        ok = bar_wait_all(&sh, &sh.s_full[w][i], s_phase >> i & 1, p.status);
        s_phase ^= 1u << i;
        if (!ok) break;
        tc_after();
        if (any_live) {
          const int valid = prefix - (first + j) * kTcKeys;
          const uint32_t s = s_of(w, i) + lanes;
          uint32_t x[2][32];
          tm_ld32(s, x[0]);
          tm_ld32(s + 32, x[1]);
          tm_wait_ld();
          if (valid < kTcKeys) {
#pragma unroll
            for (int e = 0; e < kTcKeys; ++e)
              if (e >= valid) x[e / 32][e % 32] = 0xff800000u;  // -infinity
          }
          // The weights are first taken with the maximum so far, while this
          // tile's own is found; where that has grown too much (and in an
          // item's first tile), once more.
          uint32_t h[32], g[kFull ? 32 : 1];
          unsigned long long sum;
          for (;;) {
            const float b = m == -INFINITY ? 0.f : m - Num<T>::kShift;
            const unsigned long long scale = pack2(p.scale2, p.scale2), minus = pack2(-b, -b);
            float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            sum = 0ull;
#pragma unroll
            for (int e = 0; e < kTcKeys; e += 2) {
              const float x0 = __uint_as_float(x[e / 32][e % 32]), x1 = __uint_as_float(x[e / 32][e % 32 + 1]);
              t[e & 2] = fmaxf(t[e & 2], x0);
              t[(e & 2) + 1] = fmaxf(t[(e & 2) + 1], x1);
              const float2 y = unpack2(fma2(pack2(x0, x1), scale, minus));
              const float e0 = exp2_(y.x), e1 = exp2_(y.y);
              sum = add2(sum, pack2(e0, e1));
              if (kFull) two_parts<T>(make_float2(e0, e1), h[e / 2], g[kFull ? e / 2 : 0]);
              else h[e / 2] = Num<T>::pack(e0, e1);
            }
            const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * p.scale2;
            const bool grow = top > (m == -INFINITY ? m : m + kGrow);
            if (!__any_sync(0xffffffffu, grow)) break;
            if (j == 0) {
              m = fmaxf(m, top);
              continue;
            }
            // O can be changed once the half's P V so far are complete
            ok = bar_wait_all(&sh, &sh.o_full[w], (done - 1) & 1, p.status);
            if (!ok) break;
            tc_after();
            const float f = grow ? exp2_(m - top) : 1.f;
            if (grow) m = top;
            l *= f;
            for (int q = 0; q < D / 16; ++q) {
              uint32_t y[16];
              tm_ld16(o_of(w) + lanes + q * 16, y);
              tm_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
              tm_st16(o_of(w) + lanes + q * 16, y);
            }
          }
          if (!ok) break;
          tm_st32(s, h);
          if constexpr (kFull) tm_st32(s + 32, g);
          const float2 both = unpack2(sum);
          l += both.x + both.y;
          tm_wait_st();
        }
        // The item's end waits for its last P V; a phase's parity only tells it
        // from the one before if that one is known to be complete, which it is
        // to be before the last P is handed over.
        if (j + 1 == n && done > 0) ok = bar_wait_all(&sh, &sh.o_full[w], (done - 1) & 1, p.status);
        if (!ok) break;
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.p_full[w][i]);
        ++done;
      }
      if (!ok) break;
      // ---- the partial result
      if (half_live) {
        ok = bar_wait_all(&sh, &sh.o_full[w], (done - 1) & 1, p.status);
        if (!ok) break;
        tc_after();
      }
      if (any_live) {
        const long long slot = (c + item) * 2ll + w;
        const bool again = kLong && live && item == last_item;
        m -= Num<T>::kShift;
        const Sum sum(m, l, again ? p.tc_ml[slot * kTcRows + r] : make_float2(-INFINITY, 0.f));
        for (int q = 0; q < D / 32; ++q) {
          uint32_t x[32];
          tm_ld32(o_of(w) + lanes + q * 32, x);
          tm_wait_ld();
          float4 *const to = p.tc_o + (slot * (D / 4) + q * 8) * kTcRows + r;
          if (again)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 y = to[i * kTcRows];
              x[4 * i] = __float_as_uint(sum(__uint_as_float(x[4 * i]), y.x));
              x[4 * i + 1] = __float_as_uint(sum(__uint_as_float(x[4 * i + 1]), y.y));
              x[4 * i + 2] = __float_as_uint(sum(__uint_as_float(x[4 * i + 2]), y.z));
              x[4 * i + 3] = __float_as_uint(sum(__uint_as_float(x[4 * i + 3]), y.w));
            }
          if (live)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              to[i * kTcRows] = make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]), __uint_as_float(x[4 * i + 2]),
                                            __uint_as_float(x[4 * i + 3]));
        }
        if (live) p.tc_ml[slot * kTcRows + r] = make_float2(m, l);
      }
      last_item = item;
      tc_before();
    }
  }
  __syncthreads();
  if (sh.dead) {
    // Given up: what is in flight ends before shared and tensor memory go, within
    // a second.  The matrix instructions of both halves, whichever role gave up:
    uint64_t end;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(end));
    end += 1000000000ull;
    if (warp >= 10) {
      if (elect_one()) mma_commit(&sh.drain[warp - 10]);
      __syncwarp();
      bar_wait_until(&sh.drain[warp - 10], 0, end);
    }
    // The tensor copies: an entry's phase ends with them once both copying warps
    // have arrived, so the arrivals of the one that is behind are made up for.
    if (warp == 8) {
      const int a = min(sh.sent[0], sh.sent[1]), b = max(sh.sent[0], sh.sent[1]);
      for (int e = a; e < b; ++e) bar_arrive(&sh.full[e % kRing]);
      for (int e = max(0, b - kRing); e < b; ++e) bar_wait_until(&sh.full[e % kRing], e / kRing & 1, end);
    }
    __syncthreads();
  }
  if (warp == 10) {
    tc_after();
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  }
}

// Join the partials of every row.  A block takes kJoinRows rows of one K/V head
// that follow one another in the partials, where a group of four elements of
// all rows is contiguous: each load of a warp is 4 pieces of 128 bytes.  Of its
// 16 warps, 4 share the elements and 4 the partials: lane q * 8 + i of warp
// 4 s + w adds up, for row i, element groups w * D / 16 + q + 4 k of partials
// s, s + 4, ...  The weights 2^(m - M) come first, into shared memory, while the
// first partials are on their way.  With kOne there is a block to each SM at
// most, and a thread has the registers for more of them (1B, batch 16 over 8000
// positions: 22.9 us a call against 24.8); where there are more blocks two
// share an SM (5 drafted tokens over 5003 positions, 168 blocks: 28.7 us
// against 30.4).
constexpr int kJoinRows = 8;
constexpr int kJoinThreads = 512;
constexpr int kJoinMax = 512;  // partials of a row whose weights are kept at a time
template <class T, int D, bool kFull, bool kOne>
__global__ void __launch_bounds__(kJoinThreads, kOne ? 1 : 2) join_kernel(const AttnDev p) {
  __shared__ float w_s[kJoinMax][kJoinRows], m_s[kJoinThreads / 32][kJoinRows], l_s[kJoinThreads / 32][kJoinRows];
  __shared__ float4 a_s[3][D / 4][kJoinRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ri = lane % kJoinRows;
  const int d0 = (warp & 3) * (D / 16) + lane / kJoinRows, part = warp >> 2;
  constexpr int kGroups = D / 64;  // element groups of a lane
  // partials on their way at first: as many as the registers hold (at 64 a thread
  // and D = 128, 2 and 3 spill: 1 and 2.5 of 80 us more for 64 sequences over
  // 32768 positions)
  constexpr int kAhead = kOne ? 10 / kGroups : D == 64 ? 4 : 1;
  pdl_wait();
  {
    const int kv = blockIdx.y, first = blockIdx.x * kJoinRows, row = min(first + ri, p.B * p.T * p.G - 1);
    // (small numbers: a half added, the product with the reciprocal is never off by one)
    const int u = (int)((row + 0.5f) * p.inv_G), b = (int)((u + 0.5f) * p.inv_T), g = row - u * p.G, t = u - b * p.T;
    // what every part's list says is read at once; what a row has no part in is
    // not used, whatever stands there
    const int x = t * p.G + g, item2 = p.n_prefix_items + (b * p.nkv + kv) * p.own_tiles + x / kRows;
    const int item1 = p.tc_groups ? kv * p.tc_groups + first / kTcGroup : kv * p.prefix_tiles + first / kRows;
    const int2 who1 = p.tc_groups ? p.tc_who[item1] : p.n_prefix_items ? p.who[item1] : make_int2(0, -1), who2 = p.who[item2];
    const int how = p.how[b];
    const bool live = first + ri == row && how >= 0;
    // this row's partials: n1 of the prefix, n2 of its own part
    int n1 = 0, n2 = 0;
    const float2 *ml1 = p.part_ml, *ml2 = p.part_ml;
    const float4 *o1 = p.part_o, *o2 = p.part_o;
    int ms1 = kRows, rows1 = kRows;
    if (live && (how & 1)) {
      if (p.tc_groups) {  // (a block's rows are of one half: kTcRows is a multiple of kJoinRows)
        const int in = first % kTcGroup + ri, r = in % kTcRows;
        n1 = who1.y - who1.x + 1;
        const long long half = (who1.x + item1) * 2ll + in / kTcRows;  // this row's half of each slot
        ms1 = 2 * kTcRows;
        rows1 = kTcRows;
        ml1 = p.tc_ml + half * kTcRows + r;
        o1 = p.tc_o + (half * (D / 4) + d0) * kTcRows + r;
      } else {
        const int r = row % kRows;
        n1 = who1.y - who1.x + 1;
        ml1 = p.part_ml + (long long)(who1.x + item1) * kRows + r;
        o1 = p.part_o + ((long long)(who1.x + item1) * (D / 4) + d0) * kRows + r;
      }
    }
    if (live && (how & 2)) {
      const int r = x % kRows;
      n2 = who2.y - who2.x + 1;
      ml2 = p.part_ml + (long long)(who2.x + item2) * kRows + r;
      o2 = p.part_o + ((long long)(who2.x + item2) * (D / 4) + d0) * kRows + r;
    }
    // ---- the row's maximum and sum: thread 8 k + i looks at partials k, k + 64, ... of row i
    const int n = n1 + n2;
    auto ml_of = [&](int i) {
      const float2 *y = i < n1 ? ml1 + i * (long long)ms1 : ml2 + (i - n1) * (long long)kRows;
      return *y;
    };
    // the first partials' elements are on their way while the weights are found
    const float2 y0 = tid / kJoinRows < n ? ml_of(tid / kJoinRows) : make_float2(0.f, 0.f);
    const long long step1 = (long long)ms1 * (D / 4), step2 = (long long)kRows * (D / 4);
    o2 -= n1 * step2;
    float4 z0[kAhead][kGroups];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = part + 4 * j;
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
        if (i < n) z0[j][k] = i < n1 ? o1[i * step1 + 4 * k * rows1] : o2[i * step2 + 4 * k * kRows];
    }
    float M = y0.y != 0.f ? y0.x : -INFINITY, L = 0.f;
#pragma unroll 1
    for (int i = tid / kJoinRows + kJoinThreads / kJoinRows; i < n; i += kJoinThreads / kJoinRows) {
      const float2 y = ml_of(i);
      if (y.y != 0.f) M = fmaxf(M, y.x);
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane < kJoinRows) m_s[warp][ri] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) M = fmaxf(M, m_s[w][ri]);
    const float base = M == -INFINITY ? 0.f : M;
    // ---- the elements
    float4 a[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int n_max = __reduce_max_sync(0xffffffffu, n);  // (of the block: every warp has the same rows)
#pragma unroll 1
    for (int i0 = 0; i0 < n_max; i0 += kJoinMax) {
      for (int i = i0 + tid / kJoinRows; i < min(n, i0 + kJoinMax); i += kJoinThreads / kJoinRows) {
        const float2 y = i == tid / kJoinRows ? y0 : ml_of(i);
        const float f = y.y == 0.f ? 0.f : exp2_(y.x - base);
        w_s[i - i0][ri] = f;
        L += f * y.y;
      }
      __syncthreads();
      if (i0 == 0)
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (part + 4 * j >= n) break;
          const float f = w_s[part + 4 * j][ri];
#pragma unroll
          for (int k = 0; k < kGroups; ++k) {
            a[k].x = fmaf(z0[j][k].x, f, a[k].x);
            a[k].y = fmaf(z0[j][k].y, f, a[k].y);
            a[k].z = fmaf(z0[j][k].z, f, a[k].z);
            a[k].w = fmaf(z0[j][k].w, f, a[k].w);
          }
        }
      auto add = [&](const float4 *o, long long os, int rows, int from, int to) {  // partials from, from + 4, ... of this row
#pragma unroll 4
        for (int i = from; i < to; i += 4) {
          const float f = w_s[i - i0][ri];
#pragma unroll
          for (int k = 0; k < kGroups; ++k) {
            const float4 z = o[i * os + 4 * k * rows];
            a[k].x = fmaf(z.x, f, a[k].x);
            a[k].y = fmaf(z.y, f, a[k].y);
            a[k].z = fmaf(z.z, f, a[k].z);
            a[k].w = fmaf(z.w, f, a[k].w);
          }
        }
      };
      const int from = part + (i0 == 0 ? 4 * kAhead : i0), end = min(n, i0 + kJoinMax), cut = min(max(n1, i0), end);
      add(o1, step1, rows1, from, cut);
      add(o2, step2, kRows, max(from, cut + ((part - cut) & 3)), end);
      if (i0 + kJoinMax < n_max) __syncthreads();
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane < kJoinRows) l_s[warp][ri] = L;
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
      if (part > 0) a_s[part - 1][d0 + 4 * k][ri] = a[k];
    __syncthreads();
    if (part == 0 && live) {
      L = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinThreads / 32; ++w) L += l_s[w][ri];
      const float inv = L == 0.f ? 0.f : 1.f / L;  // (a NaN stays)
      char *op = p.out + b * p.o_bs + t * p.o_ts + (kv * p.G + g) * p.o_hs + d0 * 8;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        for (int s = 0; s < 3; ++s) {
          const float4 z = a_s[s][d0 + 4 * k][ri];
          a[k].x += z.x;
          a[k].y += z.y;
          a[k].z += z.z;
          a[k].w += z.w;
        }
        if (kFull) {
          // rounded to 22 bits, the step number in the two low ones
          const unsigned tag = *p.epoch & 3u;
          auto word = [&](float x) { return ((__float_as_uint(x * inv) + 2u) & ~3u) | tag; };
          reinterpret_cast<uint4 *>(p.tagged + ((long long)b * p.nq + kv * p.G + g) * D)[d0 + 4 * k] =
              make_uint4(word(a[k].x), word(a[k].y), word(a[k].z), word(a[k].w));
          continue;
        }
        *reinterpret_cast<uint2 *>(op + k * 32) = make_uint2(Num<T>::pack(a[k].x * inv, a[k].y * inv), Num<T>::pack(a[k].z * inv, a[k].w * inv));
      }
      if (p.lse && d0 == 0)
        p.lse[((long long)b * p.T + t) * p.nq + kv * p.G + g] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
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
  const int64_t own = (int64_t)a->table_width * a->page, pre = (int64_t)a->n_prefix_pages * a->page;
  if (own >= (1ll << 31) - 64 || pre >= (1ll << 31) - 64) return MK_ERR_INVALID_ARG;
  // the work of a whole call is counted in 32 bits
  const int64_t rows = (int64_t)a->batch * a->n_tokens * (a->n_q_heads / a->n_kv_heads), tiles = rows / kRows + a->batch;
  if (a->n_kv_heads * tiles * ((own + pre) / kUnit + 2 + 2 * kItemCost) >= 1ll << 31) return MK_ERR_INVALID_ARG;
  return MK_OK;
}

// A prefix with room for this many positions (page list x page size) is taken on
// the tensor cores, a shorter one as items of the small kind.  Measured with 64
// positions of a sequence's own, in us, tensor cores / small items, at 4, 64 and
// 1024 rows a kv head:
//   8 kv heads of 64:   512: 16.0/14.1  16.5/16.1  39.0/39.4
//                      1024: 16.5/16.4  18.5/16.5  41.2/49.1
//                      4096: 18.6/24.7  20.6/20.8  51.2/102.5
//   8 kv heads of 128:  512: 17.4/14.5  19.6/18.5  47.5/48.5
//                      1024: 18.6/18.3  20.8/20.6  51.1/62.1
//                      4096: 20.7/34.1  23.2/29.0  63.6/139.5
// The number of rows hardly moves the crossing.
constexpr int kTcMinPrefix = 1024;

void fill(const mk_attn_shared_args *a, AttnDev *d) {
  d->B = a->batch;
  d->T = a->n_tokens;
  d->nq = a->n_q_heads;
  d->nkv = a->n_kv_heads;
  d->G = d->nq / d->nkv;
  const int R = d->B * d->T * d->G;
  d->tc_groups = (int64_t)a->n_prefix_pages * a->page >= kTcMinPrefix ? (R + kTcGroup - 1) / kTcGroup : 0;
  d->prefix_tiles = a->n_prefix_pages > 0 && !d->tc_groups ? (R + kRows - 1) / kRows : 0;
  d->n_prefix_items = d->nkv * d->prefix_tiles;
  d->inv_G = 1.f / (float)d->G;
  d->inv_T = 1.f / (float)d->T;
  d->own_tiles = (d->T * d->G + kRows - 1) / kRows;
  d->n_items = d->n_prefix_items + d->B * d->nkv * d->own_tiles;
}

// The tensor map of K or V: boxes of 64 elements x `rows` positions of one head
// of one page, with the 128-byte swizzle.
bool make_map(CUtensorMap *map, const mk_attn_shared_args *a, const void *x, int rows) {
  typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) != cudaSuccess ||
        how != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return (Encode)f;
  }();
  if (!encode) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)a->head_dim, (cuuint64_t)a->page, (cuuint64_t)a->n_kv_heads, (cuuint64_t)a->n_pages};
  const cuuint64_t strides[3] = {2 * (cuuint64_t)a->row_stride, 2 * (cuuint64_t)a->kv_head_stride, 2 * (cuuint64_t)a->page_stride};
  for (cuuint64_t t : strides)
    if (t == 0 || t >= 1ull << 40) return false;
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
  return encode(map, a->dtype == MK_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                const_cast<void *>(x), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The parts of the workspace: bytes of each, in order.
struct Sizes {
  int64_t part_o, part_ml, tc_o, tc_ml, who, tc_who, how;
};
Sizes sizes_of(const AttnDev &d, int head_dim, int sms) {
  const int64_t rows = ((int64_t)sms * kWarps + d.n_items) * kRows;
  const int64_t tc = d.tc_groups ? ((int64_t)sms + d.nkv * d.tc_groups) * 2 * kTcRows : 0;
  return Sizes{rows * head_dim * 4, rows * 8, tc * head_dim * 4, tc * 8, 8 * (int64_t)d.n_items, 8 * (int64_t)d.nkv * d.tc_groups, 4 * (int64_t)d.B};
}

template <class T, int D, bool kFull, bool kLong>
int launch_attn(const AttnDev &p, const CUtensorMap (&maps)[2], int sms, cudaStream_t st) {
  static_assert(smem_stages<D>() + 4 * (kMaxRowsB + 1) + 1024 <= tc_smem<D, kFull>(), "the small items' stages and sums fit");
  static std::atomic<uint64_t> allowed;
  const int rc = serve_allow_smem(allowed, (const void *)attn_kernel<T, D, kFull, kLong>, tc_smem<D, kFull>());
  return rc ? rc : serve_launch(attn_kernel<T, D, kFull, kLong>, dim3(sms), kTcThreads, tc_smem<D, kFull>(), st, false, 1, p, maps[0], maps[1]);
}

template <class T, int D, bool kFull = false>
int launch(const AttnDev &p, const CUtensorMap (&maps)[2], int sms, cudaStream_t st) {
  // Where a page list has no room for more than kMaxSum positions a block, the
  // kernel is built without the adding up (which costs the softmax warps
  // registers: 64 sequences over 32768 positions 79.3 us with it, 76.0 without).
  const int64_t tiles = (int64_t)p.n_prefix_pages * p.page / kTcKeys + 1 + kTcItemCost;
  const bool is_long = tiles * p.nkv * p.tc_groups / sms + 1 > kMaxSum / kTcKeys;
  int rc = is_long ? launch_attn<T, D, kFull, true>(p, maps, sms, st) : launch_attn<T, D, kFull, false>(p, maps, sms, st);
  if (rc) return rc;
  const dim3 grid((p.B * p.T * p.G + kJoinRows - 1) / kJoinRows, p.nkv);
  return grid.x * grid.y <= (unsigned)sms ? serve_launch(join_kernel<T, D, kFull, true>, grid, kJoinThreads, 0, st, true, 1, p)
                                          : serve_launch(join_kernel<T, D, kFull, false>, grid, kJoinThreads, 0, st, true, 1, p);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int64_t mk_attn_shared_workspace_bytes(const mk_attn_shared_args *a) {
  if (check(a)) return 0;
  AttnDev d;
  fill(a, &d);
  int sms = 0;
  if (serve_sms(&sms)) return 0;
  const Sizes z = sizes_of(d, a->head_dim, sms);
  return z.part_o + z.part_ml + z.tc_o + z.tc_ml + z.who + z.tc_who + z.how;
}

// mk_attn_shared; with `tagged`, q is an engine's buffer of tagged words
// [batch][n_q_heads][d] and the output goes to `tagged`, with the step's tag.
static int attn_shared(const mk_attn_shared_args *a, float *tagged, const unsigned *epoch, void *workspace, void *stream) {
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
  d.page_shift = (a->page & (a->page - 1)) == 0 ? __builtin_ctz((unsigned)a->page) : -1;
  d.page_units = a->page % kUnit == 0;
  d.n_prefix_pages = a->n_prefix_pages;
  d.table_width = a->table_width;
  // (never 0, so that a masked score stays -infinity)
  d.scale2 = std::max(1e-37f, (float)(std::fabs((double)a->scale) * 1.4426950408889634));
  d.flip = a->scale < 0.f ? 0x80008000u : 0u;
  int sms = 0;
  if ((rc = serve_sms(&sms))) return rc;
  const Sizes z = sizes_of(d, a->head_dim, sms);
  char *w = (char *)workspace;
  auto part = [&](int64_t bytes) {  // the sizes are multiples of 16, but for the last ones' of 8 and 4
    char *x = w;
    w += bytes;
    return x;
  };
  d.part_o = (float4 *)part(z.part_o);
  d.tc_o = (float4 *)part(z.tc_o);
  d.part_ml = (float2 *)part(z.part_ml);
  d.tc_ml = (float2 *)part(z.tc_ml);
  d.who = (int2 *)part(z.who);
  d.tc_who = (int2 *)part(z.tc_who);
  d.how = (int *)part(z.how);
  CUtensorMap maps[2] = {};
  if (d.tc_groups && d.page_units) {
    const int rows = a->page % 64 == 0 ? 64 : a->page % 32 == 0 ? 32 : 16;
    if (make_map(&maps[0], a, a->k, rows) && make_map(&maps[1], a, a->v, rows)) d.box = rows;
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (tagged) {
    d.tagged = tagged;
    d.epoch = epoch;
    d.q_bs = 4 * a->q_batch_stride;
    d.q_ts = 4 * a->q_token_stride;
    d.q_hs = 4 * a->q_head_stride;
    return a->head_dim == 64 ? launch<__nv_bfloat16, 64, true>(d, maps, sms, st) : launch<__nv_bfloat16, 128, true>(d, maps, sms, st);
  }
  if (a->dtype == MK_DTYPE_BF16)
    return a->head_dim == 64 ? launch<__nv_bfloat16, 64>(d, maps, sms, st) : launch<__nv_bfloat16, 128>(d, maps, sms, st);
  return a->head_dim == 64 ? launch<__half, 64>(d, maps, sms, st) : launch<__half, 128>(d, maps, sms, st);
}

extern "C" int mk_attn_shared(const mk_attn_shared_args *a, void *workspace, void *stream) {
  return attn_shared(a, nullptr, nullptr, workspace, stream);
}

int mk::attn_shared_tagged(const mk_attn_shared_args *a, float *out, const unsigned *epoch, void *workspace, void *stream) {
  return attn_shared(a, out, epoch, workspace, stream);
}
