// Pages of a K/V cache: resize, fork, compact and copy (include/mk_serve.h).
//
// Each call is one block that does the bookkeeping -- it holds a list entry
// per thread and the page bitmap in shared memory, and orders everything by
// prefix sums, so the result does not depend on the order of atomics -- and a
// grid-wide kernel that moves the rows the bookkeeping listed, whose blocks
// start as soon as the bookkeeping's one is done.  The bookkeeping is bound by the
// latency of its few dependent steps: 16 sequences resized in 11.6 us and 15
// forked in 10.4 us, both kernels included (captured, B200).
#include "serve_common.h"

#include <algorithm>

namespace mk {
namespace {

constexpr int kMetaThreads = 1024;  // one list entry per thread
constexpr int kMaxList = kMetaThreads;
constexpr int kMaxCopy = 16384;
constexpr int kMaxPages = 1 << 20;  // bitmap of all pages in shared memory: 128 KB

// The parts of a bookkeeping buffer.
struct State {
  int32_t *head, *len, *refs, *free_, *table;
  int n_seqs, max_pages, n_pages;
};
State state_of(const mk_kv_state &s) {
  State r;
  r.head = s.words;
  r.len = s.words + 4;
  r.refs = r.len + s.n_seqs;
  r.free_ = r.refs + s.n_pages;
  r.table = r.free_ + s.n_pages;
  r.n_seqs = s.n_seqs;
  r.max_pages = s.max_pages;
  r.n_pages = s.n_pages;
  return r;
}

// One copy of rows between pages (the entry layout of mk_kv_copy's list).
struct Job {
  int src_page, src_row, dst_page, dst_row, rows;
};
// Workspace: the number of jobs, then (64 bytes on) jobs, flags or page numbers.
struct Work {
  int *count;
  Job *jobs;
};
__host__ __device__ inline Work work_of(void *ws) {
  Work w;
  w.count = static_cast<int *>(ws);
  w.jobs = reinterpret_cast<Job *>(static_cast<char *>(ws) + 64);
  return w;
}

// Inclusive sum over the block; every thread calls it; red: 33 ints of shared memory.
__device__ int block_incl_sum(int v, int *red, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = warp_incl_sum(v);
  __syncthreads();  // red may still be read from the last call
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < (int)(blockDim.x >> 5) ? red[lane] : 0;
    red[lane] = warp_incl_sum(w);
  }
  __syncthreads();
  if (warp > 0) x += red[warp - 1];
  *total = red[31];
  return x;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }
__device__ __forceinline__ bool page_ok(const State &s, int p) { return (unsigned)p < (unsigned)s.n_pages; }
// the free stack's depth, whatever the buffer holds
__device__ __forceinline__ int depth(const State &s) { return min(max(s.head[0], 0), s.n_pages); }

// ---------------------------------------------------------------- init

__global__ void init_kernel(State s) {
  const long long n = 4ll + s.n_seqs + 2ll * s.n_pages + (long long)s.n_seqs * s.max_pages;
  const long long f0 = 4ll + s.n_seqs + s.n_pages, t0 = f0 + s.n_pages;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x)
    s.head[i] = i == 0 ? s.n_pages : i < f0 ? 0 : i < t0 ? (int)(t0 - 1 - i) : -1;
}

// ---------------------------------------------------------------- resize

__global__ void __launch_bounds__(kMetaThreads) resize_kernel(State s, const int *seqs, const int *lens, int n, int page,
                                                              void *ws) {
  extern __shared__ unsigned freed[];  // bit per page that this call frees
  __shared__ int red[33], seq_s[kMaxList], old_s[kMaxList], new_s[kMaxList], last_s[kMaxList], start_s[kMaxList];
  __shared__ int any_freed, n_jobs, oom;
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  const int words = (s.n_pages + 31) / 32;
  for (int w = i; w < words; w += kMetaThreads) freed[w] = 0;
  if (i == 0) any_freed = n_jobs = oom = 0;
  Work wk = work_of(ws);
  pdl_wait();
  int32_t *status = s.head + 1;
  const int seq = i < n ? seqs[i] : -1, want = i < n ? lens[i] : 0;
  int have = 0;
  bool ok = i < n && (unsigned)seq < (unsigned)s.n_seqs;
  if (ok) {
    have = s.len[seq];
    const long long cap = (long long)s.max_pages * page;
    ok = have >= 0 && have <= cap && want >= 0 && want <= cap;
  }
  seq_s[i] = i < n ? seq : -1;
  __syncthreads();
  for (int j = 0; ok && j < i; ++j) ok = seq_s[j] != seq;
  if (i < n && !ok) report(status, MK_ERR_DEVICE_INPUT);
  // old_s = new_s marks a skipped entry for the loops over entries below
  old_s[i] = ok ? have : 0;
  new_s[i] = ok ? want : 0;
  __syncthreads();

  // 1. give pages back: a warp per entry
  for (int e = warp; e < n; e += kMetaThreads / 32) {
    const int a = ceil_div(new_s[e], page), b = ceil_div(old_s[e], page);
    for (int j = a + lane; j < b; j += 32) {
      int32_t *t = s.table + (long long)seq_s[e] * s.max_pages + j;
      const int p = *t;
      *t = -1;
      if (!page_ok(s, p)) {
        report(status, MK_ERR_DEVICE_INPUT);
        continue;
      }
      const int was = atomicSub(s.refs + p, 1);
      if (was == 1) {
        atomicOr(freed + p / 32, 1u << (p & 31));
        any_freed = 1;
      } else if (was < 1) {  // a page that nobody held: leave it free
        atomicAdd(s.refs + p, 1);
        report(status, MK_ERR_DEVICE_INPUT);
      }
    }
  }
  __syncthreads();
  int top = depth(s);
  if (any_freed) {  // onto the stack in ascending order: a run of words per thread
    const int run = (words + kMetaThreads - 1) / kMetaThreads, w0 = min(i * run, words), w1 = min(w0 + run, words);
    int mine = 0, total;
    for (int w = w0; w < w1; ++w) mine += __popc(freed[w]);
    int at = top + block_incl_sum(mine, red, &total) - mine;
    for (int w = w0; w < w1; ++w)
      for (unsigned b = freed[w]; b; b &= b - 1, ++at)
        if (at < s.n_pages) s.free_[at] = w * 32 + __ffs(b) - 1;
    top = min(top + total, s.n_pages);
  }
  __syncthreads();

  // 2. growth.  Entry i takes `need` pages from position `start` below the top.
  const bool grows = ok && want > have;
  const int b = ceil_div(have, page), part = have % page;
  int last = -1, refs = 0;
  if (grows && part) {
    last = s.table[(long long)seq * s.max_pages + b - 1];
    if (page_ok(s, last)) {
      refs = s.refs[last];
    } else {
      report(status, MK_ERR_DEVICE_INPUT);
      last = -1;
    }
  }
  last_s[i] = last;
  __syncthreads();
  bool cow = refs > 1;
  if (cow) {  // of the entries that grow on this page, the last holder keeps it
    int before = 0;
    for (int j = 0; j < i; ++j) before += last_s[j] == last;
    cow = refs - before > 1;
  }
  // new pages of this entry; more than there are is as good as one more, and
  // kMaxList of them then add up in 32 bits
  const int more = grows ? min(ceil_div(want, page) - b, s.n_pages + 1) : 0;
  static_assert((long long)kMaxList * (kMaxPages + 2) < 1ll << 31, "sums of needed pages");
  int need = more + cow, total;
  int start = block_incl_sum(need, red, &total) - need;
  bool take = grows;
  if (total > top) {
    // Not enough pages: decide entry by entry, as the list is ordered.  A
    // skipped entry does not copy, so the next holder's turn changes with it.
    start_s[i] = grows ? more : -1;
    __syncthreads();
    if (i == 0) {
      int used = 0;
      for (int e = 0; e < n; ++e) {
        if (start_s[e] < 0) continue;
        const int p = last_s[e];
        const int c = p >= 0 && s.refs[p] > 1;
        if (used + start_s[e] + c > top) {
          start_s[e] = -1;
          oom = 1;
          continue;
        }
        if (c) s.refs[p] -= 1;
        const int k = start_s[e] + c;
        start_s[e] = used * 2 + c;
        used += k;
      }
      red[32] = used;
    }
    __syncthreads();
    total = red[32];
    take = grows && start_s[i] >= 0;
    start = take ? start_s[i] >> 1 : 0;
    cow = take && (start_s[i] & 1);
    if (i == 0 && oom) report(status, MK_ERR_OUT_OF_MEMORY);
  } else if (cow) {
    atomicSub(s.refs + last, 1);
  }
  auto pop = [&](int k) {  // the k-th page below the top
    const int p = s.free_[top - 1 - k];
    if (page_ok(s, p)) {
      s.refs[p] = 1;
      return p;
    }
    report(status, MK_ERR_DEVICE_INPUT);
    return -1;
  };
  if (cow) {
    const int p = pop(start);
    s.table[(long long)seq * s.max_pages + b - 1] = p;
    if (p >= 0) wk.jobs[atomicAdd(&n_jobs, 1)] = Job{last, 0, p, 0, part};
  }
  // an entry that does not take its pages keeps its length
  __syncthreads();
  start_s[i] = start + cow;
  if (grows && !take) new_s[i] = have;
  __syncthreads();
  for (int e = warp; e < n; e += kMetaThreads / 32) {
    const int b0 = ceil_div(old_s[e], page), a = ceil_div(new_s[e], page);
    for (int j = b0 + lane; j < a; j += 32)
      s.table[(long long)seq_s[e] * s.max_pages + j] = pop(start_s[e] + j - b0);
  }
  if (ok && (take || !grows)) s.len[seq] = want;
  if (i == 0) {
    s.head[0] = top - total;
    *wk.count = n_jobs;
  }
}

// ---------------------------------------------------------------- fork

__global__ void __launch_bounds__(kMetaThreads) fork_kernel(State s, const int *parents, const int *children, int n,
                                                            int page, void *ws) {
  __shared__ int red[33], par_s[kMaxList], kid_s[kMaxList], full_s[kMaxList];
  __shared__ int n_jobs;
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  Work wk = work_of(ws);
  if (i == 0) n_jobs = 0;
  pdl_wait();
  int32_t *status = s.head + 1;
  const int par = i < n ? parents[i] : -1, kid = i < n ? children[i] : -1;
  bool ok = i < n && (unsigned)par < (unsigned)s.n_seqs && (unsigned)kid < (unsigned)s.n_seqs && par != kid;
  int len = 0;
  if (ok) {
    len = s.len[par];
    ok = s.len[kid] == 0 && len >= 0 && len <= (long long)s.max_pages * page;
  }
  kid_s[i] = ok ? kid : -1;
  __syncthreads();
  for (int j = 0; ok && j < i; ++j) ok = kid_s[j] != kid;
  if (i < n && !ok) report(status, MK_ERR_DEVICE_INPUT);
  const int full = len / page, rem = len % page;
  int total;
  const int need = ok && rem ? 1 : 0;
  const int rank = block_incl_sum(need, red, &total) - need, top = depth(s);
  if (need && rank >= top) {
    ok = false;
    report(status, MK_ERR_OUT_OF_MEMORY);
  }
  par_s[i] = par;
  full_s[i] = ok ? full : 0;
  __syncthreads();
  // shared pages: a warp per entry
  for (int e = warp; e < n; e += kMetaThreads / 32)
    for (int j = lane; j < full_s[e]; j += 32) {
      const int p = s.table[(long long)par_s[e] * s.max_pages + j];
      s.table[(long long)kid_s[e] * s.max_pages + j] = p;
      if (page_ok(s, p)) atomicAdd(s.refs + p, 1);
      else report(status, MK_ERR_DEVICE_INPUT);
    }
  if (ok && rem) {
    const int from = s.table[(long long)par * s.max_pages + full], p = s.free_[top - 1 - rank];
    if (page_ok(s, p)) s.refs[p] = 1;
    s.table[(long long)kid * s.max_pages + full] = p;
    if (page_ok(s, from) && page_ok(s, p)) wk.jobs[atomicAdd(&n_jobs, 1)] = Job{from, 0, p, 0, rem};
    else report(status, MK_ERR_DEVICE_INPUT);
  }
  if (ok) s.len[kid] = len;
  __syncthreads();
  if (i == 0) {
    s.head[0] = top - min(total, top);
    *wk.count = n_jobs;
  }
}

// ---------------------------------------------------------------- compact

// Bookkeeping of a compaction; to[p] for p >= the pages in use: where page p
// goes (-1: nowhere).
__global__ void __launch_bounds__(kMetaThreads) compact_kernel(State s, int *to, int page, void *ws) {
  extern __shared__ unsigned live[];
  __shared__ int red[33];
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5, P = s.n_pages;
  const int words = (P + 31) / 32;
  Work wk = work_of(ws);
  pdl_wait();
  for (int w = warp; w < words; w += kMetaThreads / 32) {
    const int p = w * 32 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, p < P && s.refs[p] > 0);
    if (lane == 0) live[w] = m;
  }
  __syncthreads();
  const int run = (words + kMetaThreads - 1) / kMetaThreads, w0 = min(i * run, words), w1 = min(w0 + run, words);
  int mine = 0, n_live, n_moved;
  for (int w = w0; w < w1; ++w) mine += __popc(live[w]);
  block_incl_sum(mine, red, &n_live);
  // bits of word w that number pages below n_live
  auto low = [&](int w) {
    const int k = n_live - w * 32;
    return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1;
  };
  int holes = 0, movers = 0;
  for (int w = w0; w < w1; ++w) {
    holes += __popc(~live[w] & low(w));
    movers += __popc(live[w] & ~low(w));
  }
  int h = block_incl_sum(holes, red, &n_moved) - holes, m = block_incl_sum(movers, red, &n_moved) - movers;
  for (int w = w0; w < w1; ++w) {
    for (unsigned b = ~live[w] & low(w); b; b &= b - 1) {
      Job &j = wk.jobs[h++];
      j.dst_page = w * 32 + __ffs(b) - 1;
      j.src_row = j.dst_row = 0;
      j.rows = page;
    }
    for (unsigned b = live[w] & ~low(w); b; b &= b - 1) wk.jobs[m++].src_page = w * 32 + __ffs(b) - 1;
  }
  for (int p = n_live + i; p < P; p += kMetaThreads) to[p] = -1;
  for (int k = i; k < P - n_live; k += kMetaThreads) s.free_[k] = P - 1 - k;
  __syncthreads();
  for (int k = i; k < n_moved; k += kMetaThreads) {
    const Job j = wk.jobs[k];
    to[j.src_page] = j.dst_page;
    s.refs[j.dst_page] = s.refs[j.src_page];
    s.refs[j.src_page] = 0;
  }
  if (i == 0) {
    s.head[0] = P - n_live;
    *wk.count = n_moved;
  }
}

// ---------------------------------------------------------------- rows

struct PoolDev {
  char *k, *v;
  int n_pages, page;
};

// Entry i of a caller's list may be copied: in range, and its rows written by
// no earlier entry and read by none.  One block per entry, which looks at all the
// others (a call with entries of one row, 2 layers of 2 heads: 8.1 us for 125
// entries, 12.2 for 1024, 447 for 16384).
__global__ void __launch_bounds__(256) check_copy_kernel(const Job *items, int n, PoolDev a, PoolDev b, int *good,
                                                         int32_t *status) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const bool same = a.k == b.k;
  auto valid = [&](const Job &x) {
    return (unsigned)x.src_page < (unsigned)a.n_pages && (unsigned)x.dst_page < (unsigned)b.n_pages && x.src_row >= 0 &&
           x.dst_row >= 0 && x.rows >= 0 && x.src_row <= a.page - x.rows && x.dst_row <= b.page - x.rows;
  };
  const Job x = items[i];
  bool bad = !valid(x);
  if (!bad && x.rows > 0)
    for (int j = threadIdx.x; j < n && !bad; j += blockDim.x) {
      const Job y = items[j];
      if (y.rows <= 0 || !valid(y)) continue;
      if (j < i && y.dst_page == x.dst_page && y.dst_row < x.dst_row + x.rows && x.dst_row < y.dst_row + y.rows) bad = true;
      if (same && y.src_page == x.dst_page && y.src_row < x.dst_row + x.rows && x.dst_row < y.src_row + y.rows) bad = true;
    }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    good[i] = !bad;
    if (bad) report(status, MK_ERR_DEVICE_INPUT);
  }
}

// A 16-byte load that leaves L1 alone, and its store.
__device__ __forceinline__ uint4 ld16(const char *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

constexpr int kCopyThreads = 256;
constexpr int kPieceBytes = 8192;  // bytes of one head's rows that a warp moves at a time

// Move the listed rows: a warp takes one piece (kPieceBytes at most, contiguous
// in both pools) of one (job, layer, head, K or V) at a time.  `count` NULL:
// n jobs, those with good[i] = 0 left out.  With `to`, the blocks also
// renumber the pages of every sequence (compaction).  Bound by memory: pieces
// of 8 KB, eight 16-byte loads of a lane in flight before their stores, eight
// blocks an SM.  230 MB copied (459 MB read and written) in 79.8 us with the
// check of the list, 5.8 TB/s; 267 MB moved by a compaction in 96.0 us with its
// bookkeeping.
__global__ void __launch_bounds__(kCopyThreads) move_kernel(const Job *jobs, const int *count, int n, const int *good,
                                                            PoolDev a, PoolDev b, int n_layers, int n_heads,
                                                            int row_bytes, int piece_rows, int pieces, const int *to,
                                                            State s) {
  pdl_wait();
  if (count) n = *count;
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (kCopyThreads / 32);
  const long long warp0 = blockIdx.x * (long long)(kCopyThreads / 32) + (threadIdx.x >> 5);
  const long long per_job = (long long)n_layers * 2 * n_heads * pieces, units = per_job * n;
  for (long long u = warp0; u < units; u += warps) {
    const int job = (int)(u / per_job);
    int r = (int)(u % per_job);
    const int piece = r % pieces;
    r /= pieces;
    const int head = r % n_heads;
    r /= n_heads;
    const int layer = r >> 1;
    const bool is_v = r & 1;
    if (good && !good[job]) continue;
    const Job j = jobs[job];
    const int row = piece * piece_rows, rows = min(piece_rows, j.rows - row);
    if (rows <= 0) continue;
    const char *x = (is_v ? a.v : a.k) +
                    ((((long long)layer * a.n_pages + j.src_page) * n_heads + head) * a.page + j.src_row + row) * row_bytes;
    char *y = (is_v ? b.v : b.k) +
              ((((long long)layer * b.n_pages + j.dst_page) * n_heads + head) * b.page + j.dst_row + row) * row_bytes;
    const long long bytes = (long long)rows * row_bytes;
    long long o = lane * 16;
    for (; o + 7 * 512 < bytes; o += 8 * 512) {
      uint4 v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = ld16(x + o + q * 512);
#pragma unroll
      for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4 *>(y + o + q * 512) = v[q];
    }
    for (; o < bytes; o += 512) *reinterpret_cast<uint4 *>(y + o) = ld16(x + o);
  }
  if (to) {
    const int used = s.n_pages - s.head[0];
    const long long m = (long long)s.n_seqs * s.max_pages;
    for (long long t = blockIdx.x * (long long)kCopyThreads + threadIdx.x; t < m; t += (long long)gridDim.x * kCopyThreads) {
      const int p = s.table[t];
      if (p < used) continue;
      const int q = p < s.n_pages ? to[p] : -1;
      if (q >= 0) s.table[t] = q;
      else report(s.head + 1, MK_ERR_DEVICE_INPUT);
    }
  }
}

bool pool_ok(const mk_kv_pool *p) {
  return p && p->k && p->v && aligned_to(p->k, 16) && aligned_to(p->v, 16) && p->n_layers > 0 && p->n_pages > 0 &&
         p->n_pages <= kMaxPages && p->n_kv_heads > 0 && p->page > 0 && p->page <= (1 << 24) && p->head_dim > 0 &&
         (p->elem_bytes == 1 || p->elem_bytes == 2 || p->elem_bytes == 4) &&
         ((long long)p->head_dim * p->elem_bytes) % 16 == 0 && p->n_layers <= 65536 && p->n_kv_heads <= 65536 &&
         p->head_dim <= 65536;
}
bool state_ok(const mk_kv_state *s) {
  return s && s->words && aligned_to(s->words, 16) && s->n_seqs > 0 && s->n_seqs <= (1 << 20) && s->max_pages > 0 &&
         s->n_pages > 0 && s->n_pages <= kMaxPages;
}
size_t pool_bytes(const mk_kv_pool &p) {
  return (size_t)p.n_layers * p.n_pages * p.n_kv_heads * p.page * p.head_dim * p.elem_bytes;
}
PoolDev dev(const mk_kv_pool &p) { return PoolDev{(char *)p.k, (char *)p.v, p.n_pages, p.page}; }

// Pieces that a job's rows of one head are moved in, and warps' units of a job.
int piece_rows_of(const mk_kv_pool &p) { return std::max(1, kPieceBytes / (p.head_dim * p.elem_bytes)); }
int pieces_of(const mk_kv_pool &a, const mk_kv_pool &b) {
  return (std::min(a.page, b.page) + piece_rows_of(a) - 1) / piece_rows_of(a);
}
// They are counted in 32 bits.
bool units_ok(const mk_kv_pool &a, const mk_kv_pool &b) {
  return (long long)a.n_layers * 2 * a.n_kv_heads * pieces_of(a, b) < 1ll << 31;
}
bool both_ok(const mk_kv_pool *p, const mk_kv_state *s) {
  return pool_ok(p) && state_ok(s) && p->n_pages == s->n_pages && (long long)s->max_pages * p->page < (1ll << 31) &&
         units_ok(*p, *p);
}

// The grid that moves the listed rows (max_jobs: as many as there can be).
int launch_move(const mk_kv_pool &a, const mk_kv_pool &b, const Job *jobs, const int *count, int n, const int *good,
                const int *to, const State &s, cudaStream_t st) {
  int sms = 0, rc = serve_sms(&sms);
  if (rc) return rc;
  const int row_bytes = a.head_dim * a.elem_bytes;
  const int piece_rows = piece_rows_of(a), pieces = pieces_of(a, b);
  const long long units = (long long)a.n_layers * 2 * a.n_kv_heads * pieces * n;
  const long long blocks = (units + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  const int grid = (int)std::max<long long>(1, std::min<long long>(blocks, (long long)sms * 8));
  return serve_launch(move_kernel, dim3(grid), kCopyThreads, 0, st, true, 1, jobs, count, n, good, dev(a), dev(b),
                      a.n_layers, a.n_kv_heads, row_bytes, piece_rows, pieces, to, s);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int64_t mk_kv_state_words(int32_t n_seqs, int32_t max_pages, int32_t n_pages) {
  if (n_seqs < 1 || max_pages < 1 || n_pages < 1) return 0;
  return 4 + (int64_t)n_seqs + 2 * (int64_t)n_pages + (int64_t)n_seqs * max_pages;
}

extern "C" int64_t mk_kv_workspace_bytes(int32_t n_pages, int32_t n) {
  if (n_pages < 1 || n < 0) return 0;
  // jobs of a list or of a compaction, the page map, the list's flags
  const int64_t jobs = std::max<int64_t>(n_pages, n);
  return (64 + jobs * (int64_t)sizeof(Job) + 4 * jobs + 255) / 256 * 256;
}

extern "C" int mk_kv_init(const mk_kv_state *st, void *stream) {
  if (!state_ok(st)) return MK_ERR_INVALID_ARG;
  const long long n = mk_kv_state_words(st->n_seqs, st->max_pages, st->n_pages);
  const int grid = (int)std::min<long long>((n + 255) / 256, 1184);
  return serve_launch(init_kernel, dim3(grid), 256, 0, (cudaStream_t)stream, false, 1, state_of(*st));
}

extern "C" int mk_kv_resize(const mk_kv_pool *pool, const mk_kv_state *st, const int32_t *seqs, const int32_t *lens,
                            int32_t n, void *workspace, void *stream) {
  if (!both_ok(pool, st) || !seqs || !lens || n < 1 || n > kMaxList || !workspace || !aligned_to(workspace, 256))
    return MK_ERR_INVALID_ARG;
  cudaStream_t cs = (cudaStream_t)stream;
  const State s = state_of(*st);
  const size_t smem = ((size_t)st->n_pages + 31) / 32 * 4;
  static std::atomic<uint64_t> allowed;
  int rc = smem > 16384 ? serve_allow_smem(allowed, (const void *)resize_kernel, kMaxPages / 8) : MK_OK;
  if (!rc) rc = serve_launch(resize_kernel, dim3(1), kMetaThreads, smem, cs, false, 1, s, seqs, lens, n, pool->page, workspace);
  if (rc) return rc;
  const Work w = work_of(workspace);
  return launch_move(*pool, *pool, w.jobs, w.count, n, nullptr, nullptr, s, cs);
}

extern "C" int mk_kv_fork(const mk_kv_pool *pool, const mk_kv_state *st, const int32_t *parents,
                          const int32_t *children, int32_t n, void *workspace, void *stream) {
  if (!both_ok(pool, st) || !parents || !children || n < 1 || n > kMaxList || !workspace || !aligned_to(workspace, 256))
    return MK_ERR_INVALID_ARG;
  cudaStream_t cs = (cudaStream_t)stream;
  const State s = state_of(*st);
  int rc = serve_launch(fork_kernel, dim3(1), kMetaThreads, 0, cs, false, 1, s, parents, children, n, pool->page, workspace);
  if (rc) return rc;
  const Work w = work_of(workspace);
  return launch_move(*pool, *pool, w.jobs, w.count, n, nullptr, nullptr, s, cs);
}

extern "C" int mk_kv_compact(const mk_kv_pool *pool, const mk_kv_state *st, void *workspace, void *stream) {
  if (!both_ok(pool, st) || !workspace || !aligned_to(workspace, 256)) return MK_ERR_INVALID_ARG;
  cudaStream_t cs = (cudaStream_t)stream;
  const State s = state_of(*st);
  const Work w = work_of(workspace);
  int *to = reinterpret_cast<int *>(w.jobs + st->n_pages);
  const size_t smem = ((size_t)st->n_pages + 31) / 32 * 4;
  static std::atomic<uint64_t> allowed;
  int rc = smem > 16384 ? serve_allow_smem(allowed, (const void *)compact_kernel, kMaxPages / 8) : MK_OK;
  if (!rc) rc = serve_launch(compact_kernel, dim3(1), kMetaThreads, smem, cs, false, 1, s, to, pool->page, workspace);
  if (rc) return rc;
  return launch_move(*pool, *pool, w.jobs, w.count, st->n_pages, nullptr, to, s, cs);
}

extern "C" int mk_kv_copy(const mk_kv_pool *src, const mk_kv_pool *dst, const int32_t *items, int32_t n,
                          int32_t *status, void *workspace, void *stream) {
  if (!pool_ok(src) || !pool_ok(dst) || !items || n < 1 || n > kMaxCopy || !workspace || !aligned_to(workspace, 256))
    return MK_ERR_INVALID_ARG;
  if (src->n_layers != dst->n_layers || src->n_kv_heads != dst->n_kv_heads || src->head_dim != dst->head_dim ||
      src->elem_bytes != dst->elem_bytes || !units_ok(*src, *dst))
    return MK_ERR_INVALID_ARG;
  const bool same = src->k == dst->k && src->v == dst->v && src->n_pages == dst->n_pages && src->page == dst->page;
  if (!same) {  // else every pair of buffers is apart
    const char *xs[] = {(const char *)src->k, (const char *)src->v}, *ys[] = {(const char *)dst->k, (const char *)dst->v};
    const size_t nx = pool_bytes(*src), ny = pool_bytes(*dst);
    for (const char *x : xs)
      for (const char *y : ys)
        if (x < y + ny && y < x + nx) return MK_ERR_INVALID_ARG;
  }
  cudaStream_t cs = (cudaStream_t)stream;
  int *good = reinterpret_cast<int *>(static_cast<char *>(workspace) + 64);
  const Job *jobs = reinterpret_cast<const Job *>(items);
  int rc = serve_launch(check_copy_kernel, dim3(n), 256, 0, cs, false, 1, jobs, n, dev(*src), dev(*dst), good, status);
  if (rc) return rc;
  return launch_move(*src, *dst, jobs, nullptr, n, good, nullptr, State{}, cs);
}
