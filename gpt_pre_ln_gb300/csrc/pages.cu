// Bookkeeping of a paged key-value cache, all of it on the device so that a
// serving loop can be captured into a graph: page table rows shared between
// sequences (refs[p] = table entries that name page p, 0 = free), pages handed
// out lowest id first, copy on write of a shared page, compaction, and the
// keys and values of new tokens stored in their pages.
//
// Only the copies move data worth counting (a page of GPT-2 small with 16
// positions holds 590 KB); they are bound by HBM bandwidth.  The table work is
// integers, decided in a fixed order, so that results do not depend on timing;
// it is bound by the latency of a few dependent loads.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace gpt2 {

namespace {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int warp_incl(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// Exclusive prefix sum over the block (whole warps); *total = the block's
// sum.  s: one int per warp.  Ends with a barrier after the last read of s.
__device__ __forceinline__ int block_excl(int v, int* s, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int incl = warp_incl(v, lane);
  if (lane == 31) s[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int x = lane < warps ? s[lane] : 0;
    const int y = warp_incl(x, lane);
    s[lane] = y - x;
    if (lane == 31) s[32] = y;
  }
  __syncthreads();
  const int r = s[warp] + incl - v;
  *total = s[32];
  __syncthreads();
  return r;
}

// ---------------------------------------------------------------- free
// Entries of the given rows go to -1 and their pages lose a reference.  With
// keep_first and keep_last both 0 the whole row goes and its length becomes
// -1; otherwise pages that hold one of the first keep_first or last keep_last
// positions, or positions at or behind the length, stay.
// A row named twice, or out of range, leaves everything as it was.
__device__ __forceinline__ bool rows_distinct(const int32_t* rows, int n, int n_seq, unsigned* s_mark) {
  // s_mark: one bit per row, (n_seq + 31) / 32 words
  bool bad = false;
  for (int i = threadIdx.x; i < (n_seq + 31) / 32; i += blockDim.x) s_mark[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int r = rows[i];
    if (r < 0 || r >= n_seq)
      bad = true;
    else if (atomicOr(&s_mark[r >> 5], 1u << (r & 31)) & (1u << (r & 31)))
      bad = true;
  }
  return !__syncthreads_or(bad);
}

__device__ __forceinline__ void drop_ref(int32_t* refs, int page, int n_pages, unsigned* err) {
  if (page >= n_pages) {
    record_error(err, kErrRange, kSitePagedPage);
    return;
  }
  atomicSub(&refs[page], 1);
}

__global__ void __launch_bounds__(256) pages_free(int32_t* table, int32_t* lens, int32_t* refs,
                                                  const int32_t* __restrict__ rows, int n, int n_seq, int max_pages,
                                                  int page_size, int n_pages, int keep_first, int keep_last,
                                                  unsigned* err) {
  __shared__ unsigned s_mark[kMaxPagedSeqs / 32];
  griddep_wait();
  griddep_launch_dependents();
  if (!rows_distinct(rows, n, n_seq, s_mark)) {
    if (threadIdx.x == 0) record_error(err, kErrRange, kSitePagedRow);
    return;
  }
  const bool all = keep_first == 0 && keep_last == 0;
  const int row = rows[blockIdx.x];
  const int len = all ? 0 : lens[row];
  if (!all && len < 0) return;
  int32_t* t = table + static_cast<long long>(row) * max_pages;
  for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < max_pages; c += gridDim.y * blockDim.x) {
    const int p = t[c];
    if (p < 0) continue;
    const int first = c * page_size;
    if (!all && (first < keep_first || first + page_size > len - keep_last)) continue;
    drop_ref(refs, p, n_pages, err);
    t[c] = -1;
  }
  if (all && blockIdx.y == 0 && threadIdx.x == 0) lens[row] = -1;
}

// ---------------------------------------------------------------- fork
// Row children[i] takes the pages that hold the positions of row parents[i]
// (as all rows were before the call) and its length; what it named before
// loses a reference.  One CTA (5.5 us for 8 rows of 64 pages, the cluster 6.9),
// or with many entries one cluster of eight: each
// CTA owns a set of columns and reads them for every pair before it writes
// any; the lengths are read by every CTA before the cluster's barrier and
// written after it.
constexpr int kForkCtas = 8;
constexpr int kForkThreads = 512;
constexpr int kForkEntries = 8192;  // of all pairs at a time: 1024 pairs by 8 columns at least

__global__ void __launch_bounds__(kForkThreads) pages_fork(int32_t* table, int32_t* lens, int32_t* refs,
                                                           const int32_t* __restrict__ parents,
                                                           const int32_t* __restrict__ children, int n, int n_seq,
                                                           int max_pages, int page_size, int n_pages, unsigned* err) {
  __shared__ unsigned s_mark[kMaxPagedSeqs / 32];
  __shared__ int s_new[kForkEntries];
  __shared__ int s_len[kMaxPagedSeqs];
  griddep_wait();
  griddep_launch_dependents();
  const int rank = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += kForkThreads) {
    const int p = parents[i];
    bad |= p < 0 || p >= n_seq;
    s_len[i] = p >= 0 && p < n_seq ? lens[p] : -1;
  }
  const bool ok = rows_distinct(children, n, n_seq, s_mark) && !__syncthreads_or(bad);
  if (ctas > 1) cluster_sync();  // every CTA has read the lengths
  if (!ok) {
    if (threadIdx.x == 0) record_error(err, kErrRange, kSitePagedRow);
    return;
  }
  if (rank == 0)
    for (int i = threadIdx.x; i < n; i += kForkThreads) lens[children[i]] = s_len[i];
  const int cols = min(max_pages, kForkEntries / n);
  for (int c0 = rank * cols; c0 < max_pages; c0 += ctas * cols) {
    for (int k = threadIdx.x; k < n * cols; k += kForkThreads) {
      const int i = k / cols, c = c0 + k % cols;
      int p = -1;
      if (c < max_pages && static_cast<long long>(c) * page_size < s_len[i])
        p = table[static_cast<long long>(parents[i]) * max_pages + c];
      if (p >= 0) {
        if (p < n_pages) {
          atomicAdd(&refs[p], 1);
        } else {
          record_error(err, kErrRange, kSitePagedPage);
          p = -1;
        }
      }
      s_new[k] = p;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < n * cols; k += kForkThreads) {
      const int i = k / cols, c = c0 + k % cols;
      if (c >= max_pages) continue;
      int32_t* at = table + static_cast<long long>(children[i]) * max_pages + c;
      const int old = *at;
      if (old >= 0) drop_ref(refs, old, n_pages, err);
      *at = s_new[k];
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- reserve
struct ReserveWs {
  int* head;     // [0] copies to make
  int3* copies;  // source page, target page, positions
  int* fresh;    // pages handed out, in order
  int* left;     // the page each of them replaces, or -1
  int* writers;  // [n_pages] rows of this call that write to a shared page
  int* last;     // [n_pages] and the last entry among them
};

// One CTA, bound by the latency of its loads.  The entries that the new positions lens[b] .. lens[b] + n_new[b] -
// 1 of every row need, laid end to end (row by row), are shared out to the
// threads.  An entry gets the next free page (lowest id first) when it has
// none, or when other rows hold its page too: of the rows that write to one
// page in this call the last keeps it if nobody else reads it.
// Counting writers with atomics and taking the highest index keeps the choice
// independent of timing.
// Anything out of range, or too few free pages, leaves everything as it was.
__global__ void __launch_bounds__(kPlanThreads) pages_reserve(int32_t* table, const int32_t* __restrict__ lens,
                                                              int32_t* refs, const int32_t* __restrict__ n_new,
                                                              int n_seq, int max_pages, int page_size, int n_pages,
                                                              ReserveWs ws, unsigned* err) {
  __shared__ int s_scan[33];
  __shared__ int s_base[kMaxPagedSeqs + 1], s_col[kMaxPagedSeqs];
  __shared__ __align__(16) int s_page[kPlanThreads];
  __shared__ int s_fresh[kPlanThreads];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  // the first pages' counts, on their way from the start
  int low[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) low[i] = tid * 8 + i < n_pages ? refs[tid * 8 + i] : 1;
  // columns of each row (one row per thread: n_seq <= kPlanThreads)
  int cols = 0, bad = 0;
  if (tid < n_seq) {
    const int len = lens[tid], add = n_new[tid];
    if (len >= 0 && add > 0) {
      if (static_cast<long long>(len) + add > static_cast<long long>(max_pages) * page_size) {
        bad = 1;
      } else {
        s_col[tid] = len / page_size;
        cols = (len + add - 1) / page_size - len / page_size + 1;
      }
    }
  }
  if (tid == 0) ws.head[0] = 0;
  int total;
  const int base = block_excl(cols, s_scan, &total);
  if (tid < n_seq) s_base[tid] = base;
  if (tid == 0) s_base[n_seq] = total;
  if (__syncthreads_or(bad)) {
    if (tid == 0) record_error(err, kErrRange, kSitePagedLength);
    return;
  }
  auto where = [&](int k, int& b, int& c) {
    int lo = 0, hi = n_seq;  // last b with base[b] <= k
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_base[mid] <= k)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
    c = s_col[lo] + k - s_base[lo];
  };
  if (total <= kPlanThreads) {
    // One entry per thread (a decode step, short prompts): everything stays in
    // registers and shared memory, two rounds of loads in all (5.7 us for nine
    // sequences; the general way below 8.9).
    const bool mine = tid < total;
    int b = 0, c = 0, p = -1, r = 0;
    if (mine) {
      where(tid, b, c);
      p = table[static_cast<long long>(b) * max_pages + c];
      if (p >= n_pages)
        bad = 1;
      else if (p >= 0)
        r = refs[p];
    }
    const int held_here = mine ? min(max(lens[b] - c * page_size, 0), page_size) : 0;
    s_page[tid] = r > 1 ? p : -1;
    if (__syncthreads_or(bad)) {
      if (tid == 0) record_error(err, kErrRange, kSitePagedPage);
      return;
    }
    bool take = mine && p < 0;
    if (r > 1) {
      int writers = 0, last = 0;
      for (int k = 0; k < total; k += 4) {
        const int4 q = *reinterpret_cast<const int4*>(&s_page[k]);
        const int same[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (same[e] == p) {
            ++writers;
            last = k + e;
          }
      }
      take = !(writers == r && last == tid);
    }
    const int held = take && p >= 0 ? held_here : 0;
    int both;  // takers, and 2^16 times copies
    const int at2 = block_excl((take ? 1 : 0) + (held > 0 ? 1 << 16 : 0), s_scan, &both);
    const int want = both & 0xffff;
    int found = 0;
    for (int p0 = 0; found < want && p0 < n_pages; p0 += kPlanThreads * 8) {
      if (p0 > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int q = p0 + tid * 8 + i;
          low[i] = q < n_pages ? refs[q] : 1;
        }
      }
      int n = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) n += low[i] == 0 ? 1 : 0;
      int got;
      int at = found + block_excl(n, s_scan, &got);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (low[i] == 0) {
          if (at < want) s_fresh[at] = p0 + tid * 8 + i;
          ++at;
        }
      found += got;
    }
    if (found < want) {
      if (tid == 0) record_error(err, kErrRange, kSitePagedFull);
      return;
    }
    __syncthreads();
    if (take) {
      const int fresh = s_fresh[at2 & 0xffff];
      table[static_cast<long long>(b) * max_pages + c] = fresh;
      refs[fresh] = 1;
      if (p >= 0) atomicSub(&refs[p], 1);
      if (held > 0) ws.copies[at2 >> 16] = make_int3(p, fresh, held);
    }
    if (tid == 0) ws.head[0] = both >> 16;
    return;
  }
  // shared pages: who writes to them
  bool shared_any = false;
  for (int k = tid; k < total; k += kPlanThreads) {
    int b, c;
    where(k, b, c);
    const int p = table[static_cast<long long>(b) * max_pages + c];
    if (p < 0) continue;
    if (p >= n_pages) {
      bad = 1;
    } else if (refs[p] > 1) {
      ws.writers[p] = 0;
      ws.last[p] = -1;
      shared_any = true;
    }
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) record_error(err, kErrRange, kSitePagedPage);
    return;
  }
  if (__syncthreads_or(shared_any)) {
    for (int k = tid; k < total; k += kPlanThreads) {
      int b, c;
      where(k, b, c);
      const int p = table[static_cast<long long>(b) * max_pages + c];
      if (p >= 0 && refs[p] > 1) {
        atomicAdd(&ws.writers[p], 1);
        atomicMax(&ws.last[p], k);
      }
    }
    __syncthreads();
  }
  auto wants = [&](int k, int b, int c) {
    const int p = table[static_cast<long long>(b) * max_pages + c];
    if (p < 0) return true;
    if (refs[p] <= 1) return false;
    return !(ws.writers[p] == refs[p] && ws.last[p] == k);
  };
  int need = 0;
  for (int k = tid; k < total; k += kPlanThreads) {
    int b, c;
    where(k, b, c);
    need += wants(k, b, c) ? 1 : 0;
  }
  int want;
  block_excl(need, s_scan, &want);
  if (want == 0) return;
  // the lowest free pages, in order
  int found = 0;
  for (int p0 = 0; p0 < n_pages && found < want; p0 += kPlanThreads * 8) {
    const int q = p0 + tid * 8;
    int r[8];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r[i] = q + i < n_pages ? refs[q + i] : 1;
      mine += r[i] == 0 ? 1 : 0;
    }
    int got;
    int at = found + block_excl(mine, s_scan, &got);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r[i] == 0) {
        if (at < want) ws.fresh[at] = q + i;
        ++at;
      }
    found += got;
  }
  if (found < want) {
    if (tid == 0) record_error(err, kErrRange, kSitePagedFull);
    return;
  }
  __syncthreads();
  // hand them out in the order of the entries
  int given = 0, copies = 0;
  for (int k0 = 0; k0 < total; k0 += kPlanThreads) {
    const int k = k0 + tid;
    int b = 0, c = 0, p = -1;
    bool take = false;
    if (k < total) {
      where(k, b, c);
      take = wants(k, b, c);
      p = table[static_cast<long long>(b) * max_pages + c];
    }
    // positions of the old page that hold something
    const int held = take && p >= 0 ? min(max(lens[b] - c * page_size, 0), page_size) : 0;
    int n_take, n_copy;
    const int at = given + block_excl(take ? 1 : 0, s_scan, &n_take);
    const int cat = copies + block_excl(held > 0 ? 1 : 0, s_scan, &n_copy);
    if (take) {
      const int fresh = ws.fresh[at];
      table[static_cast<long long>(b) * max_pages + c] = fresh;
      refs[fresh] = 1;
      ws.left[at] = p;
      if (held > 0) ws.copies[cat] = make_int3(p, fresh, held);
    }
    given += n_take;
    copies += n_copy;
  }
  if (tid == 0) ws.head[0] = copies;
  // the pages left behind lose their references only now: the decisions above
  // read the counts as they were
  __syncthreads();
  for (int i = tid; i < want; i += kPlanThreads)
    if (ws.left[i] >= 0) atomicSub(&refs[ws.left[i]], 1);
}

// ---------------------------------------------------------------- copies
// Positions 0 .. rows-1 of page src to page dst, for head[0] copies: rows *
// 128 contiguous bytes for each of the chunks = n_layer * 2 * n_kv_head
// pieces of a page.  One warp per piece, four 16-byte loads of a lane in
// flight.  No page is the source of one copy and the target of another.
// Bound by HBM: 360 pages of 1.5 MB take 172 us, 6.6 TB/s, 98% of what a plain
// copy reaches.
constexpr int kCopyThreads = 256;
__device__ __forceinline__ void copy_rows(uint4* pages, int n, const int3* copies, int chunks, int page_size) {
  const int lane = threadIdx.x & 31;
  const long long units = static_cast<long long>(n) * chunks;
  const int step = gridDim.x * (kCopyThreads / 32);
  const long long chunk_vecs = page_size * 8;
  for (long long u = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
    const int i = static_cast<int>(u / chunks), c = static_cast<int>(u - static_cast<long long>(i) * chunks);
    const int3 job = copies[i];
    const uint4* src = pages + (static_cast<long long>(job.x) * chunks + c) * chunk_vecs;
    uint4* dst = pages + (static_cast<long long>(job.y) * chunks + c) * chunk_vecs;
    const int vecs = job.z * 8;
    for (int v = lane; v < vecs; v += 128) {
      uint4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v + 32 * e < vecs) x[e] = src[v + 32 * e];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v + 32 * e < vecs) dst[v + 32 * e] = x[e];
    }
  }
}
__global__ void __launch_bounds__(kCopyThreads) pages_copy(uint4* pages, const int* __restrict__ head,
                                                           const int3* __restrict__ copies, int chunks,
                                                           int page_size) {
  griddep_wait();
  griddep_launch_dependents();
  copy_rows(pages, *head, copies, chunks, page_size);
}

// ---------------------------------------------------------------- compact
// U pages are in use.  The f-th free page below U takes the contents of the
// page that is f-th in use from the end; there are as many of those at or
// above U as there are free ones below it.  With before(i) pages in use below
// page i, a free page i < U is number i - before(i) and a page in use is
// number U - 1 - before(i) from the end, so one pass of counts per block and
// one of ranks place everything.
constexpr int kScanThreads = 256;
constexpr int kScanPer = 16;
constexpr int kScanPages = kScanThreads * kScanPer;  // pages per block
struct CompactWs {
  int* head;     // [0] moves
  int3* copies;  // [moves]
  int* target;   // [n_pages]: new id of a page at or above U, -1 if not in use
  int* counts;   // pages in use per block
};

__global__ void __launch_bounds__(kScanThreads) compact_count(const int32_t* __restrict__ refs, int n_pages,
                                                              CompactWs ws) {
  __shared__ int s_scan[33];
  griddep_wait();
  griddep_launch_dependents();
  const int p0 = blockIdx.x * kScanPages;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kScanPer; ++i) {
    const int p = p0 + i * kScanThreads + threadIdx.x;
    mine += p < n_pages && refs[p] > 0 ? 1 : 0;
  }
  int total;
  block_excl(mine, s_scan, &total);
  if (threadIdx.x == 0) ws.counts[blockIdx.x] = total;
  if (blockIdx.x == 0 && threadIdx.x == 0) ws.head[0] = 0;
}

// `alone`: one CTA holds all pages and counts for itself.
__global__ void __launch_bounds__(kPlanThreads) compact_rank(const int32_t* __restrict__ refs, int n_pages,
                                                             int page_size, int32_t* n_used, bool alone, CompactWs ws) {
  __shared__ int s_scan[33];
  griddep_wait();
  griddep_launch_dependents();
  const int q = (blockIdx.x * blockDim.x + threadIdx.x) * kScanPer;
  bool on[kScanPer];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kScanPer; ++i) {
    on[i] = q + i < n_pages && refs[q + i] > 0;
    mine += on[i] ? 1 : 0;
  }
  int below = 0, all = 0;
  if (!alone)
    for (int k = threadIdx.x; k < static_cast<int>(gridDim.x); k += blockDim.x) {
      const int c = ws.counts[k];
      all += c;
      if (k < static_cast<int>(blockIdx.x)) below += c;
    }
  int total, used, before = 0;
  int rank = block_excl(mine, s_scan, &total);
  if (alone) {
    used = total;
  } else {
    block_excl(all, s_scan, &used);
    block_excl(below, s_scan, &before);
    rank += before;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_used = used;
  int holes = 0;
#pragma unroll
  for (int i = 0; i < kScanPer; ++i) {
    const int p = q + i;
    if (p >= n_pages) break;
    if (p < used && !on[i]) {
      ws.copies[p - rank].y = p;
      ws.copies[p - rank].z = page_size;
      ++holes;
    }
    if (p >= used) {
      ws.target[p] = on[i] ? used - 1 - rank : -1;  // number of its copy, for now
      if (on[i]) ws.copies[used - 1 - rank].x = p;
    }
    rank += on[i] ? 1 : 0;
  }
  int sum;
  block_excl(holes, s_scan, &sum);
  if (threadIdx.x == 0) {
    if (alone)
      ws.head[0] = sum;
    else if (sum)
      atomicAdd(ws.head, sum);
  }
}

// The tables and counts after the moves, then the moves.
__global__ void __launch_bounds__(kCopyThreads) compact_move(int32_t* table, long long entries, int32_t* refs,
                                                             int n_pages, const int32_t* __restrict__ n_used,
                                                             CompactWs ws, uint4* pages, int chunks, int page_size,
                                                             unsigned* err) {
  griddep_wait();
  griddep_launch_dependents();
  const int used = *n_used, moves = ws.head[0];
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long t0 = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (long long i = t0; i < entries; i += step) {
    const int p = table[i];
    if (p < used) continue;
    const int f = p < n_pages ? ws.target[p] : -1;
    if (f < 0) {  // names a page that does not exist or that nobody counted
      record_error(err, kErrRange, kSitePagedPage);
      continue;
    }
    table[i] = ws.copies[f].y;
  }
  for (long long f = t0; f < moves; f += step) {
    const int3 job = ws.copies[f];
    refs[job.y] = refs[job.x];
    refs[job.x] = 0;
  }
  copy_rows(pages, moves, ws.copies, chunks, page_size);
}

// ---------------------------------------------------------------- write
// Row b * T + t of k and v (n_kv heads of 64) to position lens[b] + t of
// sequence b, for t < n_new[b] (all T when n_new is null; with from_zero only of
// sequences of length 0).  ROWS rows per CTA, a thread's 16-byte pieces of all
// of them on their way at once: with 8, a head's rows of one page go out as 1 KB
// together.  Bound by HBM: 16 prompts of 512 to 1023 tokens at 25 heads take
// 26 us, 5.7 TB/s (one row per CTA 40 us, four 27, sixteen 35).
constexpr int kWriteRows = 8;
template <int ROWS>
__global__ void __launch_bounds__(512) pages_write(uint4* __restrict__ layer_pages, long long page_vecs,
                                                   const uint4* __restrict__ k, const uint4* __restrict__ v,
                                                   long long ld_vecs, const int32_t* __restrict__ table,
                                                   const int32_t* __restrict__ lens,
                                                   const int32_t* __restrict__ refs,
                                                   const int32_t* __restrict__ n_new, int T, long long rows, int n_kv,
                                                   int page_size, int max_pages, int n_pages, bool from_zero,
                                                   unsigned* err) {
  __shared__ long long s_to[ROWS];  // first vector of the row's position in its page, -1: nowhere
  griddep_wait();
  griddep_launch_dependents();
  const long long row0 = static_cast<long long>(blockIdx.x) * ROWS;
  if (threadIdx.x < ROWS) {
    const long long row = row0 + threadIdx.x;
    long long to = -1;
    if (row < rows) {
      const int b = static_cast<int>(row / T), t = static_cast<int>(row % T);
      const int len = lens[b];
      if ((from_zero ? len == 0 : len >= 0) && (!n_new || t < n_new[b])) {
        const long long pos = static_cast<long long>(len) + t;
        if (pos < static_cast<long long>(max_pages) * page_size) {
          const int c = static_cast<int>(pos / page_size);
          const int page = table[static_cast<long long>(b) * max_pages + c];
          if (page < 0 || page >= n_pages)
            record_error(err, kErrRange, kSitePagedPage);
          else if (refs[page] > 1)
            record_error(err, kErrRange, kSitePagedShared);
          else
            to = page * page_vecs + (pos - static_cast<long long>(c) * page_size) * 8;
        } else {
          record_error(err, kErrRange, kSitePagedLength);
        }
      }
    }
    s_to[threadIdx.x] = to;
  }
  __syncthreads();
  const int row_vecs = n_kv * 8;
  for (int i = threadIdx.x; i < 2 * row_vecs; i += blockDim.x) {
    const int part = i >= row_vecs ? 1 : 0;
    const int x = i - part * row_vecs;
    const uint4* from = (part ? v : k) + row0 * ld_vecs + x;
    uint4* at = layer_pages + (static_cast<long long>(part) * n_kv + (x >> 3)) * page_size * 8 + (x & 7);
    uint4 val[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (s_to[r] >= 0) val[r] = from[r * ld_vecs];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (s_to[r] >= 0) at[s_to[r]] = val[r];
  }
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
int scan_blocks(const gpt2_paged_cache* c) { return (c->n_pages + kScanPages - 1) / kScanPages; }
int copy_chunks(const gpt2_paged_cache* c) { return c->n_layer * 2 * c->n_kv_head; }

}  // namespace

size_t pages_workspace(const gpt2_paged_cache* c) {
  const size_t per_page = align256(static_cast<size_t>(c->n_pages) * 4);
  // head, the copies, and four numbers per page (reserve) or the ranks and
  // block counts (compact)
  return 256 + align256(static_cast<size_t>(c->n_pages) * sizeof(int3)) + 4 * per_page;
}

cudaError_t launch_pages_free(const gpt2_paged_cache* c, const int32_t* rows, int n, int keep_first, int keep_last,
                              cudaStream_t s) {
  const unsigned y = static_cast<unsigned>((c->max_pages + 255) / 256);
  return launch_pdl(pages_free, dim3(n, y < 64 ? y : 64), 256, 0, s, 0, c->table, c->lens, c->refs, rows, n, c->n_seq,
                    c->max_pages, c->page_size, c->n_pages, keep_first, keep_last, device_error_word());
}

cudaError_t launch_pages_fork(const gpt2_paged_cache* c, const int32_t* parents, const int32_t* children, int n,
                              cudaStream_t s) {
  const unsigned ctas = static_cast<long long>(n) * c->max_pages > kForkEntries ? kForkCtas : 1;
  return launch_pdl(pages_fork, ctas, kForkThreads, 0, s, ctas > 1 ? ctas : 0, c->table, c->lens, c->refs, parents,
                    children, n, c->n_seq, c->max_pages, c->page_size, c->n_pages, device_error_word());
}

cudaError_t launch_pages_reserve(const gpt2_paged_cache* c, const int32_t* n_new, void* ws, cudaStream_t s) {
  const size_t per_page = align256(static_cast<size_t>(c->n_pages) * 4);
  char* p = static_cast<char*>(ws);
  ReserveWs w;
  w.head = reinterpret_cast<int*>(p);
  w.copies = reinterpret_cast<int3*>(p + 256);
  p += 256 + align256(static_cast<size_t>(c->n_pages) * sizeof(int3));
  w.fresh = reinterpret_cast<int*>(p);
  w.left = reinterpret_cast<int*>(p + per_page);
  w.writers = reinterpret_cast<int*>(p + 2 * per_page);
  w.last = reinterpret_cast<int*>(p + 3 * per_page);
  cudaError_t e = launch_pdl(pages_reserve, 1, kPlanThreads, 0, s, 0, c->table, c->lens, c->refs, n_new, c->n_seq,
                             c->max_pages, c->page_size, c->n_pages, w, device_error_word());
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_copy, num_sms() * 8, kCopyThreads, 0, s, 0, static_cast<uint4*>(c->pages), w.head, w.copies,
                    copy_chunks(c), c->page_size);
}

cudaError_t launch_pages_compact(const gpt2_paged_cache* c, int32_t* n_used, void* ws, cudaStream_t s) {
  const size_t per_page = align256(static_cast<size_t>(c->n_pages) * 4);
  char* p = static_cast<char*>(ws);
  CompactWs w;
  w.head = reinterpret_cast<int*>(p);
  w.copies = reinterpret_cast<int3*>(p + 256);
  p += 256 + align256(static_cast<size_t>(c->n_pages) * sizeof(int3));
  w.target = reinterpret_cast<int*>(p);
  w.counts = reinterpret_cast<int*>(p + per_page);
  cudaError_t e;
  if (c->n_pages <= kPlanThreads * kScanPer) {
    // (6 us alone, 8.5 as two launches)
    e = launch_pdl(compact_rank, 1, kPlanThreads, 0, s, 0, c->refs, c->n_pages, c->page_size, n_used, true, w);
  } else {
    const int blocks = scan_blocks(c);
    e = launch_pdl(compact_count, blocks, kScanThreads, 0, s, 0, c->refs, c->n_pages, w);
    if (e != cudaSuccess) return e;
    e = launch_pdl(compact_rank, blocks, kScanThreads, 0, s, 0, c->refs, c->n_pages, c->page_size, n_used, false, w);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(compact_move, num_sms() * 8, kCopyThreads, 0, s, 0, c->table,
                    static_cast<long long>(c->n_seq) * c->max_pages, c->refs, c->n_pages, n_used, w,
                    static_cast<uint4*>(c->pages), copy_chunks(c), c->page_size, device_error_word());
}

cudaError_t launch_pages_write(const gpt2_paged_cache* c, int layer, const void* k, const void* v, int64_t ldkv,
                               int T, const int32_t* n_new, cudaStream_t s, bool from_zero) {
  const long long layer_vecs = 2ll * c->n_kv_head * c->page_size * 8;
  const int threads = std::min(512, (2 * c->n_kv_head * 8 + 31) / 32 * 32);
  const long long rows = static_cast<long long>(c->n_seq) * T;
  // (one row per CTA until there are more rows than CTAs fit at a time)
  const bool many = rows > 4ll * num_sms();
  const unsigned grid = static_cast<unsigned>(many ? (rows + kWriteRows - 1) / kWriteRows : rows);
  return launch_pdl(many ? pages_write<kWriteRows> : pages_write<1>, grid, threads, 0, s, 0,
                    static_cast<uint4*>(c->pages) + layer * layer_vecs, layer_vecs * c->n_layer,
                    static_cast<const uint4*>(k), static_cast<const uint4*>(v), static_cast<long long>(ldkv / 8),
                    c->table, c->lens, c->refs, n_new, T, rows, c->n_kv_head, c->page_size, c->max_pages, c->n_pages,
                    from_zero, device_error_word());
}

}  // namespace gpt2
