// Pages of a paged cache: reserve, fork, free, compact, copy.
//
// Who owns which page is decided on the device, so nothing here waits for the host.  Reserve, fork
// and compact are two launches each: a plan by one CTA (it checks the request, scans the reference
// counts for free pages, lowest first, and writes its decisions to the workspace), then a grid that
// carries it out (slots, table rows, page copies), launched as a programmatic dependent of the plan.
// One CTA is enough for the plan: it walks the counts twice, 4 bytes per page (to count, then to rank: 64 KB
// each for a pool of 16K pages), and compact's also writes 4 bytes per page.
//
// The copies are bound by memory: the bytes of a page are read and written once, in 16-byte loads,
// four in flight per thread.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "tq_internal.h"
#include "tq_launch.h"

namespace tq {
namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int COPY_THREADS = 256;
constexpr int CHUNK = COPY_THREADS * 4 * 16;   // bytes of one copy item
constexpr int CTAS_PER_SM = 8;
constexpr int MAX_CACHES = 64;                 // pools of one launch (their pointers are parameters)
constexpr unsigned FULL = 0xffffffffu;

// ------------------------------------------------------------------------------------- workspace
// int32 words: [0] pages to copy (compact: pages in use), [1] the plan's go-ahead, [2] compact: pages in
// use that stay; then the arrays below.
struct Ws {
  int32_t* head;
  int32_t* need;   // [n + 1] pages before entry i
  int32_t* tok;    // [n + 1] new tokens before entry i
  int32_t* old;    // [n] length before the call
  int32_t* mark;   // [n_seq]
  int32_t* room;   // [num_pages] free pages in order
  int32_t* from;   // [max(n, num_pages)] copy pairs
  int32_t* to;
  int32_t* map;    // [num_pages] the page, or -1 - its place in from[] (compact)
};
__host__ __device__ inline size_t ws_words(int n, int n_seq, int pages) {
  const size_t pairs = n > pages ? n : pages;
  return 16 + 2 * ((size_t)n + 1) + n + (size_t)n_seq + 2 * (size_t)pages + 2 * pairs;
}
__host__ __device__ inline Ws ws_at(int32_t* w, int n, int n_seq, int pages) {
  Ws s;
  const size_t pairs = n > pages ? n : pages;
  s.head = w;
  s.need = w + 16;
  s.tok = s.need + n + 1;
  s.old = s.tok + n + 1;
  s.mark = s.old + n;
  s.room = s.mark + n_seq;
  s.map = s.room + pages;
  s.from = s.map + pages;
  s.to = s.from + pairs;
  return s;
}

// ------------------------------------------------------------------------------------- block scan
// Exclusive prefix sum of one value per thread of a 1024-thread CTA, and the CTA's total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t& total) {
  __shared__ int64_t part[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous scan's partial sums are read
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int64_t own = part[lane];
    int64_t p = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(FULL, p, o);
      if (lane >= o) p += y;
    }
    part[lane] = p - own;
    if (lane == 31) part[32] = p;
  }
  __syncthreads();
  total = part[32];
  return part[warp] + x - v;
}

// A plan's warps take contiguous shares of the pages, a lane a page, so that a ballot ranks 32 of them and
// one scan over the warps' counts the rest.  (Chunks of 4096 pages in turn, a scan each, took 18 us for 16K
// pages; contiguous pages per thread, whose loads and stores do not coalesce, 22 us.)
constexpr int PLAN_WARPS = PLAN_THREADS / 32;
struct PageShare {
  int begin, rounds;  // first page and rounds of 32 pages
  __device__ __forceinline__ explicit PageShare(int pages) {
    rounds = (pages + 32 * PLAN_WARPS - 1) / (32 * PLAN_WARPS);
    begin = (int)(threadIdx.x >> 5) * rounds * 32;
  }
  // f(p, used, ballot of used) for every round, the whole warp together (used is false past the last page)
  template <typename F>
  __device__ __forceinline__ void each(const int32_t* refs, int pages, F&& f) const {
    const int lane = threadIdx.x & 31;
    for (int r0 = 0; r0 < rounds; r0 += 8) {
      int v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // eight rounds' loads together
        const int64_t p = (int64_t)begin + 32 * (r0 + j) + lane;
        v[j] = r0 + j < rounds && p < pages ? refs[p] : 0;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (r0 + j < rounds) {
          const unsigned m = __ballot_sync(FULL, v[j] > 0);
          f((int64_t)begin + 32 * (r0 + j) + lane, v[j] > 0, m);
        }
    }
  }
};
__device__ __forceinline__ int below_lane(unsigned m) { return __popc(m & ((1u << (threadIdx.x & 31)) - 1u)); }
// Exclusive prefix sum over the warps of a count that is the same in all lanes, and its total.
__device__ __forceinline__ int64_t warp_counts(int n, int64_t& total) {
  const int lane = threadIdx.x & 31;
  const int64_t at = block_scan(lane == 0 ? n : 0, total);
  return __shfl_sync(FULL, at, 0);
}

// The first `need` free pages in order to room[]; returns how many free pages there are.
__device__ int64_t free_pages(const tq_page_table& pt, int64_t need, int32_t* room) {
  const PageShare share(pt.num_pages);
  auto is_free = [&](int64_t p, unsigned used) {  // free pages of the round, without those past the last page
    const int64_t first = p - (threadIdx.x & 31);
    const unsigned real = first + 32 <= pt.num_pages ? FULL : first >= pt.num_pages ? 0u : (1u << (pt.num_pages - first)) - 1u;
    return ~used & real;
  };
  int mine = 0;
  share.each(pt.refs, pt.num_pages, [&](int64_t p, bool, unsigned m) { mine += __popc(is_free(p, m)); });
  int64_t total;
  int64_t at = warp_counts(mine, total);
  if (mine && at < need)
    share.each(pt.refs, pt.num_pages, [&](int64_t p, bool, unsigned m) {
      const unsigned f = is_free(p, m);
      const int64_t r = at + below_lane(f);
      if (((f >> (threadIdx.x & 31)) & 1u) && r < need) room[r] = (int32_t)p;
      at += __popc(f);
    });
  return total;
}

// The entry i of a list whose prefix sums are off[0..n] that holds unit u: the last i with off[i] <= u
// among those of nonzero size.
__device__ __forceinline__ int entry_of(const int32_t* off, int n, int u) {
  int lo = 0, hi = n;  // off[lo] <= u < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int ps) { return tokens / ps + (tokens % ps ? 1 : 0); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// ------------------------------------------------------------------------------------- reserve

__global__ void __launch_bounds__(PLAN_THREADS)
    reserve_plan(const tq_page_table pt, const int32_t* seqs, const int32_t* grow, int n, int n_slots, bool has_slots,
                 int32_t* wsp) {
  const Ws w = ws_at(wsp, n, pt.n_seq, pt.num_pages);
  __shared__ int bad;
  const int tid = threadIdx.x, ps = pt.page_size;
  pdl_launch();
  if (tid == 0) bad = 0;
  for (int i = tid; i < pt.n_seq; i += PLAN_THREADS) w.mark[i] = 0;
  __syncthreads();
  int64_t need = 0, toks = 0;
  for (int base = 0; base < n; base += PLAN_THREADS) {
    const int i = base + tid;
    int pg = 0, a = 0, L = 0, err = 0;
    if (i < n) {
      const int s = seqs[i];
      a = grow[i];
      if (s < 0 || s >= pt.n_seq) err = TQ_PAGES_BAD_INDEX;
      else {
        if (atomicAdd(&w.mark[s], 1) != 0) err |= TQ_PAGES_BAD_INDEX;
        L = pt.seq_lens[s];
        const int64_t most = (int64_t)pt.max_pages * ps;
        if (a < 0 || L < 0 || (int64_t)L + a > most) err |= TQ_PAGES_BAD_LENGTH;
        else {
          pg = pages_of(L + a, ps) - pages_of(L, ps);
          if (a > 0 && L % ps) {  // the first new rows go into a page that must be this sequence's alone
            const int p = pt.table[(int64_t)s * pt.max_pages + L / ps];
            if (p < 0 || p >= pt.num_pages) err |= TQ_PAGES_BAD_INDEX;
            else if (pt.refs[p] > 1) err |= TQ_PAGES_SHARED;
          }
        }
      }
      if (err) {
        atomicOr(&bad, err);
        pg = 0;
        a = 0;
      }
    }
    int64_t tp, tt;
    const int64_t bp = need + block_scan(pg, tp), bt = toks + block_scan(a, tt);
    need += tp;
    toks += tt;
    // (a sum past 32 bits is refused below, before these offsets are used)
    if (i < n) {
      w.need[i] = (int32_t)bp;
      w.tok[i] = (int32_t)bt;
      w.old[i] = L;
    }
  }
  if (tid == 0) {
    w.need[n] = (int32_t)need;
    w.tok[n] = (int32_t)toks;
    if (toks > INT_MAX || (has_slots && toks > n_slots)) bad |= TQ_PAGES_BAD_LENGTH;
  }
  __syncthreads();
  if (!bad) {
    const int64_t found = need > pt.num_pages ? 0 : free_pages(pt, need, w.room);
    if (tid == 0 && found < need) bad = TQ_PAGES_NO_ROOM;
  }
  __syncthreads();
  if (tid == 0) {
    w.head[1] = bad == 0;
    if (bad) atomicOr(pt.status, bad);
  }
}

// The new pages' table entries and counts, the new lengths and the slots.
__global__ void __launch_bounds__(COPY_THREADS)
    reserve_apply(const tq_page_table pt, const int32_t* seqs, const int32_t* grow, int n, int32_t* slots, int n_slots, int32_t* wsp) {
  const Ws w = ws_at(wsp, n, pt.n_seq, pt.num_pages);
  pdl_wait();
  const bool ok = w.head[1] != 0;
  const int toks = ok ? w.tok[n] : 0, need = ok ? w.need[n] : 0, ps = pt.page_size;
  const int first = blockIdx.x * COPY_THREADS + threadIdx.x, step = gridDim.x * COPY_THREADS;
  for (int u = first; u < need; u += step) {
    const int i = entry_of(w.need, n, u), p = w.room[u];
    pt.table[(int64_t)seqs[i] * pt.max_pages + pages_of(w.old[i], ps) + u - w.need[i]] = p;
    pt.refs[p] = 1;
  }
  for (int i = first; ok && i < n; i += step) pt.seq_lens[seqs[i]] = w.old[i] + grow[i];
  for (int64_t k = first; k < n_slots; k += step) {
    const int t = (int)k;
    int v = -1;
    if (t < toks) {
      const int i = entry_of(w.tok, n, t), pos = w.old[i] + t - w.tok[i], page = pos / ps;
      const int fresh = page - pages_of(w.old[i], ps);  // >= 0: one of the new pages; -1: the old last one
      v = (fresh >= 0 ? w.room[w.need[i] + fresh] : pt.table[(int64_t)seqs[i] * pt.max_pages + page]) * ps + (pos - page * ps);
    }
    slots[t] = v;
  }
}

// ------------------------------------------------------------------------------------- page copies

struct CopyArgs {
  uint8_t* arr[MAX_CACHES][6];
  uint32_t bytes[6];   // of a page in each array
  int chunk0[7];       // chunks of a page before each array
  int n_caches;
};

// Items (pair, cache, chunk of a page) of the pairs from[i] -> to[i], spread over the grid.
// `pages`, `status`: check the numbers of a list the caller gave (0: the plan made the list).
__device__ __forceinline__ void copy_pairs(const CopyArgs& a, const int32_t* from, const int32_t* to, int n_pairs,
                                           int pages, int32_t* status) {
  const int C = a.chunk0[6], per = C * a.n_caches;
  const int64_t items = (int64_t)n_pairs * per;
  const int tid = threadIdx.x;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int pair = (int)(item / per);
    const int r = (int)(item - (int64_t)pair * per);
    const int cache = r / C, chunk = r - cache * C;
    const int s = from[pair], d = to[pair];
    if (pages && ((unsigned)s >= (unsigned)pages || (unsigned)d >= (unsigned)pages)) {
      if (status && tid == 0 && r == 0) atomicOr(status, TQ_PAGES_BAD_INDEX);
      continue;
    }
    if (s == d) continue;
    int k = 0;
#pragma unroll
    for (int j = 1; j < 6; ++j) k = chunk >= a.chunk0[j] ? j : k;
    const uint32_t at = (uint32_t)(chunk - a.chunk0[k]) * CHUNK, len = min((uint32_t)CHUNK, a.bytes[k] - at);
    const uint4* src = reinterpret_cast<const uint4*>(a.arr[cache][k] + (int64_t)s * a.bytes[k] + at);
    uint4* dst = reinterpret_cast<uint4*>(a.arr[cache][k] + (int64_t)d * a.bytes[k] + at);
    const uint32_t nv = len / 16;
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (tid + j * COPY_THREADS < nv) v[j] = src[tid + j * COPY_THREADS];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (tid + j * COPY_THREADS < nv) dst[tid + j * COPY_THREADS] = v[j];
  }
}

__global__ void __launch_bounds__(COPY_THREADS) copy_list(const __grid_constant__ CopyArgs a, const int32_t* from,
                                                          const int32_t* to, int n, int pages, int32_t* status) {
  copy_pairs(a, from, to, n, pages, status);
}

// ------------------------------------------------------------------------------------- fork

__global__ void __launch_bounds__(PLAN_THREADS)
    fork_plan(const tq_page_table pt, const int32_t* src, const int32_t* dst, int n, int32_t* wsp) {
  const Ws w = ws_at(wsp, n, pt.n_seq, pt.num_pages);
  __shared__ int bad;
  const int tid = threadIdx.x, ps = pt.page_size;
  pdl_launch();
  if (tid == 0) bad = 0;
  for (int i = tid; i < pt.n_seq; i += PLAN_THREADS) w.mark[i] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += PLAN_THREADS) {
    const int d = dst[i];
    if (d < 0 || d >= pt.n_seq || atomicAdd(&w.mark[d], 1) != 0) atomicOr(&bad, TQ_PAGES_BAD_INDEX);
    else if (pt.seq_lens[d] != 0) atomicOr(&bad, TQ_PAGES_NOT_EMPTY);
  }
  __syncthreads();
  int64_t need = 0;
  for (int base = 0; base < n; base += PLAN_THREADS) {
    const int i = base + tid;
    int part = 0, L = 0;
    if (i < n) {
      const int s = src[i];
      if (s < 0 || s >= pt.n_seq) atomicOr(&bad, TQ_PAGES_BAD_INDEX);
      else if (*reinterpret_cast<volatile int32_t*>(&w.mark[s]) != 0) atomicOr(&bad, TQ_PAGES_NOT_EMPTY);
      else {
        L = pt.seq_lens[s];
        if (L < 0 || (int64_t)L > (int64_t)pt.max_pages * ps) {
          atomicOr(&bad, TQ_PAGES_BAD_LENGTH);
          L = 0;
        }
        part = L % ps ? 1 : 0;
        if (part) {
          const int p = pt.table[(int64_t)s * pt.max_pages + L / ps];
          if (p < 0 || p >= pt.num_pages) atomicOr(&bad, TQ_PAGES_BAD_INDEX);
        }
      }
    }
    int64_t total;
    const int64_t at = need + block_scan(part, total);
    need += total;
    if (i < n) {
      w.need[i] = (int32_t)at;
      w.old[i] = L;
    }
  }
  __syncthreads();
  if (!bad) {
    const int64_t found = need > pt.num_pages ? 0 : free_pages(pt, need, w.room);
    if (tid == 0 && found < need) bad = TQ_PAGES_NO_ROOM;
  }
  __syncthreads();
  if (tid == 0) {
    w.head[0] = bad ? 0 : (int32_t)need;
    w.head[1] = bad == 0;
    w.need[n] = (int32_t)need;
    if (bad) atomicOr(pt.status, bad);
  }
  if (bad) return;
  for (int i = tid; i < n; i += PLAN_THREADS) {
    if (w.old[i] % ps == 0) continue;
    const int r = w.need[i], p = w.room[r];
    w.from[r] = pt.table[(int64_t)src[i] * pt.max_pages + w.old[i] / ps];
    w.to[r] = p;
    pt.refs[p] = 1;
  }
}

// Table rows (when `rows`: the first of several launches), then the copies of the last pages.
__global__ void __launch_bounds__(COPY_THREADS)
    fork_apply(const tq_page_table pt, const int32_t* src, const int32_t* dst, int n, bool rows,
               const __grid_constant__ CopyArgs a, int32_t* wsp) {
  const Ws w = ws_at(wsp, n, pt.n_seq, pt.num_pages);
  pdl_wait();
  if (w.head[1] == 0) return;
  const int ps = pt.page_size;
  for (int i = blockIdx.x; rows && i < n; i += gridDim.x) {
    const int32_t* from = pt.table + (int64_t)src[i] * pt.max_pages;
    int32_t* to = pt.table + (int64_t)dst[i] * pt.max_pages;
    const int L = w.old[i], full = L / ps;
    for (int c = threadIdx.x; c < full; c += COPY_THREADS) {
      const int p = from[c];
      to[c] = p;
      if ((unsigned)p < (unsigned)pt.num_pages) atomicAdd(&pt.refs[p], 1);
      else atomicOr(pt.status, TQ_PAGES_BAD_INDEX);
    }
    if (threadIdx.x == 0) {
      if (L % ps) to[full] = w.to[w.need[i]];
      pt.seq_lens[dst[i]] = L;
    }
  }
  copy_pairs(a, w.from, w.to, w.head[0], 0, nullptr);
}

// ------------------------------------------------------------------------------------- free

// One CTA per listed sequence; the one that takes the length away frees the pages.
__global__ void __launch_bounds__(COPY_THREADS) free_seqs(const tq_page_table pt, const int32_t* seqs) {
  __shared__ int len;
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= pt.n_seq) {
    if (threadIdx.x == 0) atomicOr(pt.status, TQ_PAGES_BAD_INDEX);
    return;
  }
  if (threadIdx.x == 0) len = atomicExch(&pt.seq_lens[s], 0);
  __syncthreads();
  const int held = len <= 0 ? 0 : min(pages_of(len, pt.page_size), pt.max_pages);
  if (threadIdx.x == 0 && (len < 0 || pages_of(len, pt.page_size) > pt.max_pages)) atomicOr(pt.status, TQ_PAGES_BAD_LENGTH);
  int32_t* row = pt.table + (int64_t)s * pt.max_pages;
  for (int c = threadIdx.x; c < held; c += COPY_THREADS) {
    const int p = row[c];
    row[c] = -1;
    if ((unsigned)p < (unsigned)pt.num_pages) {
      if (atomicSub(&pt.refs[p], 1) > 0) continue;
      atomicAdd(&pt.refs[p], 1);  // nobody held it: a table that does not match the counts
    }
    atomicOr(pt.status, TQ_PAGES_BAD_INDEX);
  }
}

// ------------------------------------------------------------------------------------- compact

__global__ void __launch_bounds__(PLAN_THREADS) compact_plan(const tq_page_table pt, int32_t* wsp) {
  const Ws w = ws_at(wsp, 0, pt.n_seq, pt.num_pages);
  const int tid = threadIdx.x, P = pt.num_pages;
  pdl_launch();
  const PageShare share(P);
  int mine = 0;
  share.each(pt.refs, P, [&](int64_t, bool, unsigned m) { mine += __popc(m); });
  int64_t live;
  int n = (int)warp_counts(mine, live);  // pages in use before the share, then before the round
  // Free numbers below `live` to to[], in order; pages in use to from[], at their rank among all in use:
  // the j-th mover is from[below + j], below (head[2]) the number of pages in use below `live`.
  share.each(pt.refs, P, [&](int64_t p, bool used, unsigned m) {
    const int rank = n + below_lane(m);  // pages in use before p
    if (p < P) {
      int to = (int)p;
      if (used && p >= live) {
        w.from[rank] = (int32_t)p;
        to = -1 - rank;
      } else if (!used && p < live) {
        w.to[p - rank] = (int32_t)p;
      }
      w.map[p] = to;
      if (p == live) w.head[2] = rank;
    }
    n += __popc(m);
  });
  if (tid == 0) {
    w.head[0] = (int32_t)live;
    if (live == P) w.head[2] = P;
  }
}

__global__ void __launch_bounds__(COPY_THREADS)
    compact_apply(const tq_page_table pt, bool rows, const __grid_constant__ CopyArgs a, int32_t* wsp) {
  const Ws w = ws_at(wsp, 0, pt.n_seq, pt.num_pages);
  pdl_wait();
  const int below = w.head[2], moved = w.head[0] - below;
  if (moved == 0) return;
  for (int i = blockIdx.x * COPY_THREADS + threadIdx.x; rows && i < moved; i += gridDim.x * COPY_THREADS) {
    pt.refs[w.to[i]] = pt.refs[w.from[below + i]];
    pt.refs[w.from[below + i]] = 0;
  }
  const int64_t entries = (int64_t)pt.n_seq * pt.max_pages;
  for (int64_t i = (int64_t)blockIdx.x * COPY_THREADS + threadIdx.x; rows && i < entries;
       i += (int64_t)gridDim.x * COPY_THREADS) {
    const int p = pt.table[i];
    if ((unsigned)p >= (unsigned)pt.num_pages) continue;
    const int q = w.map[p];
    if (q < 0) pt.table[i] = w.to[-1 - q - below];
  }
  copy_pairs(a, w.from + below, w.to, moved, 0, nullptr);
}

// ------------------------------------------------------------------------------------- host

tq_status check_table(const tq_page_table* pt) {
  if (!pt) return fail(TQ_ERR_INVALID_ARG, "page table is NULL");
  if (pt->n_seq < 1 || pt->max_pages < 1 || pt->num_pages < 1)
    return fail(TQ_ERR_INVALID_ARG, "page table n_seq=%d max_pages=%d num_pages=%d", pt->n_seq, pt->max_pages, pt->num_pages);
  if (pt->page_size < 16 || pt->page_size % 16)
    return fail(TQ_ERR_INVALID_ARG, "page_size %d (a multiple of 16)", pt->page_size);
  if ((int64_t)pt->max_pages * pt->page_size > INT_MAX || (int64_t)pt->num_pages * pt->page_size > INT_MAX)
    return fail(TQ_ERR_INVALID_ARG, "a sequence or the pool holds more than 2^31 - 1 tokens");
  if (!pt->table || !pt->seq_lens || !pt->refs || !pt->status)
    return fail(TQ_ERR_INVALID_ARG, "page table array is NULL");
  if (!aligned16(pt->refs) || !aligned4(pt->table) || !aligned4(pt->seq_lens) || !aligned4(pt->status))
    return fail(TQ_ERR_INVALID_ARG, "page table arrays misaligned (refs: 16 bytes)");
  return TQ_OK;
}

tq_status check_list(const void* p, int n, const char* name) {
  if (n < 0) return fail(TQ_ERR_INVALID_ARG, "n %d", n);
  if (n > 0 && (!p || !aligned4(p))) return fail(TQ_ERR_INVALID_ARG, "%s NULL or misaligned", name);
  return TQ_OK;
}

tq_status check_pools(const tq_cache* c, int n) {
  if (n < 0) return fail(TQ_ERR_INVALID_ARG, "n_caches %d", n);
  if (n > 0 && !c) return fail(TQ_ERR_INVALID_ARG, "caches is NULL");
  for (int i = 0; i < n; ++i) {
    const tq_status st = check_pool(c + i);
    if (st != TQ_OK) return st;
    if (c[i].B != c->B || c[i].Hkv != c->Hkv || c[i].T_cap != c->T_cap || c[i].k_bits != c->k_bits ||
        c[i].v_bits != c->v_bits || c[i].qjl_m != c->qjl_m)
      return fail(TQ_ERR_INVALID_ARG, "cache %d differs in size from cache 0", i);
  }
  return TQ_OK;
}

tq_status check_pools_of(const tq_page_table* pt, const tq_cache* c, int n) {
  const tq_status st = check_pools(c, n);
  if (st != TQ_OK) return st;
  if (n > 0 && (c->B != pt->num_pages || c->T_cap != pt->page_size))
    return fail(TQ_ERR_INVALID_ARG, "pools of %d pages of %d tokens, page table of %d of %d", c->B, c->T_cap,
                pt->num_pages, pt->page_size);
  return TQ_OK;
}

CopyArgs copy_args(const tq_cache* c, int n) {
  CopyArgs a = {};
  a.n_caches = n;
  if (n == 0) return a;
  const uint32_t rows = (uint32_t)c->Hkv * c->T_cap;
  const uint32_t row[6] = {16u * c->k_bits, c->qjl_m ? 16u : 0u, 4u, c->qjl_m ? 4u : 0u, 16u * c->v_bits, 4u};
  for (int k = 0; k < 6; ++k) {
    a.bytes[k] = rows * row[k];
    a.chunk0[k + 1] = a.chunk0[k] + (int)((a.bytes[k] + CHUNK - 1) / CHUNK);
  }
  for (int i = 0; i < n; ++i) {
    uint8_t* arr[6] = {c[i].k_codes, c[i].k_signs, reinterpret_cast<uint8_t*>(c[i].k_norm),
                       reinterpret_cast<uint8_t*>(c[i].k_rnorm), c[i].v_codes, reinterpret_cast<uint8_t*>(c[i].v_norm)};
    for (int k = 0; k < 6; ++k) a.arr[i][k] = arr[k];
  }
  return a;
}

// CTAs of a launch with `items` units of work, at most all that can be resident.
int grid_for(int64_t items) { return (int)std::max<int64_t>(1, std::min<int64_t>(items, (int64_t)sm_count() * CTAS_PER_SM)); }

// A kernel that carries out the plan before it.
template <typename... K, typename... A>
tq_status launch_after(void (*kernel)(K...), int grid, cudaStream_t s, const char* name, const A&... args) {
  return launch(kernel, grid, COPY_THREADS, 0, s, true, name, args...);
}

tq_status launched(const char* name) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  return TQ_OK;
}

tq_status check_ws(const tq_page_table* pt, int n, const void* ws, size_t bytes) {
  if (!ws || !aligned16(ws)) return fail(TQ_ERR_INVALID_ARG, "workspace NULL or misaligned");
  const size_t need = tq_pages_workspace_size(pt, n);
  if (bytes < need) return fail(TQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", bytes, need);
  return TQ_OK;
}

}  // namespace
}  // namespace tq

extern "C" size_t tq_pages_workspace_size(const tq_page_table* pt, int n) {
  if (!pt || n < 0 || pt->n_seq < 1 || pt->num_pages < 1) return 0;
  return 4 * tq::ws_words(n, pt->n_seq, pt->num_pages);
}

extern "C" tq_status tq_pages_reserve(const tq_page_table* pt, const int32_t* seqs, const int32_t* new_tokens, int n,
                                      int32_t* slots, int n_slots, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  using namespace tq;
  const NvtxRange nvtx_range("tq_pages_reserve");
  clear_error();
  tq_status st = check_table(pt);
  if (st == TQ_OK) st = check_list(seqs, n, "seqs");
  if (st == TQ_OK) st = check_list(new_tokens, n, "new_tokens");
  if (st != TQ_OK) return st;
  if (n_slots < 0 || (n_slots > 0 && (!slots || !aligned4(slots))))
    return fail(TQ_ERR_INVALID_ARG, "n_slots %d, or slots NULL or misaligned", n_slots);
  st = check_ws(pt, n, workspace, workspace_bytes);
  if (st != TQ_OK || (n == 0 && n_slots == 0)) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t* w = reinterpret_cast<int32_t*>(workspace);
  reserve_plan<<<1, PLAN_THREADS, 0, s>>>(*pt, seqs, new_tokens, n, n_slots, slots != nullptr, w);
  st = launched("reserve plan");
  if (st != TQ_OK) return st;
  // (the number of new pages is known to the device alone: at most all of the pool)
  const int64_t items = std::max<int64_t>(n_slots, std::min<int64_t>(pt->num_pages, (int64_t)n * pt->max_pages));
  return launch_after(reserve_apply, grid_for((std::max<int64_t>(items, n) + COPY_THREADS - 1) / COPY_THREADS), s, "reserve", *pt, seqs,
                      new_tokens, n, slots, n_slots, w);
}

extern "C" tq_status tq_pages_fork(const tq_page_table* pt, const int32_t* src, const int32_t* dst, int n,
                                   const tq_cache* caches, int n_caches, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  using namespace tq;
  const NvtxRange nvtx_range("tq_pages_fork");
  clear_error();
  tq_status st = check_table(pt);
  if (st == TQ_OK) st = check_list(src, n, "src");
  if (st == TQ_OK) st = check_list(dst, n, "dst");
  if (st == TQ_OK) st = check_pools_of(pt, caches, n_caches);
  if (st == TQ_OK) st = check_ws(pt, n, workspace, workspace_bytes);
  if (st != TQ_OK || n == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t* w = reinterpret_cast<int32_t*>(workspace);
  fork_plan<<<1, PLAN_THREADS, 0, s>>>(*pt, src, dst, n, w);
  st = launched("fork plan");
  for (int c = 0; st == TQ_OK && (c == 0 || c < n_caches); c += MAX_CACHES) {
    const CopyArgs a = copy_args(caches + c, std::min(MAX_CACHES, n_caches - c));
    const int64_t items = std::max<int64_t>(n, (int64_t)n * a.n_caches * a.chunk0[6]);
    st = launch_after(fork_apply, grid_for(items), s, "fork", *pt, src, dst, n, c == 0, a, w);
  }
  return st;
}

extern "C" tq_status tq_pages_free(const tq_page_table* pt, const int32_t* seqs, int n, void* stream) {
  using namespace tq;
  const NvtxRange nvtx_range("tq_pages_free");
  clear_error();
  tq_status st = check_table(pt);
  if (st == TQ_OK) st = check_list(seqs, n, "seqs");
  if (st != TQ_OK || n == 0) return st;
  free_seqs<<<n, COPY_THREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(*pt, seqs);
  return launched("free");
}

extern "C" tq_status tq_pages_compact(const tq_page_table* pt, const tq_cache* caches, int n_caches, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  using namespace tq;
  const NvtxRange nvtx_range("tq_pages_compact");
  clear_error();
  tq_status st = check_table(pt);
  if (st == TQ_OK) st = check_pools_of(pt, caches, n_caches);
  if (st == TQ_OK) st = check_ws(pt, 0, workspace, workspace_bytes);
  if (st != TQ_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t* w = reinterpret_cast<int32_t*>(workspace);
  compact_plan<<<1, PLAN_THREADS, 0, s>>>(*pt, w);
  st = launched("compact plan");
  for (int c = 0; st == TQ_OK && (c == 0 || c < n_caches); c += MAX_CACHES) {
    const CopyArgs a = copy_args(caches + c, std::min(MAX_CACHES, n_caches - c));
    const int64_t rows = ((int64_t)pt->n_seq * pt->max_pages + COPY_THREADS - 1) / COPY_THREADS;
    const int64_t items = std::max<int64_t>(rows, (int64_t)(pt->num_pages / 2 + 1) * a.n_caches * a.chunk0[6]);
    st = launch_after(compact_apply, grid_for(items), s, "compact", *pt, c == 0, a, w);
  }
  return st;
}

extern "C" tq_status tq_pages_copy(const tq_cache* caches, int n_caches, const int32_t* src, const int32_t* dst, int n,
                                   int32_t* status, void* stream) {
  using namespace tq;
  const NvtxRange nvtx_range("tq_pages_copy");
  clear_error();
  tq_status st = check_list(src, n, "src");
  if (st == TQ_OK) st = check_list(dst, n, "dst");
  if (st == TQ_OK) st = check_pools(caches, n_caches);
  if (st == TQ_OK && !aligned4(status)) st = fail(TQ_ERR_INVALID_ARG, "status misaligned");
  if (st != TQ_OK || n == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for (int c = 0; st == TQ_OK && c < n_caches; c += MAX_CACHES) {
    const CopyArgs a = copy_args(caches + c, std::min(MAX_CACHES, n_caches - c));
    copy_list<<<grid_for((int64_t)n * a.n_caches * a.chunk0[6]), COPY_THREADS, 0, s>>>(a, src, dst, n, caches->B, status);
    st = launched("page copy");
  }
  return st;
}
