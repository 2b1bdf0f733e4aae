// The two ends of a step of speculative decoding: the embedding of the drafted
// tokens, and which of them stay, with their keys and values moved together in
// the paged cache.
//
// The walk starts at token 0 and goes to the first child that is the token
// chosen behind the one it stands at, until there is none.  Token path[j] then
// stands for position len + j: in every layer its K and V go from place
// len + path[j] to place len + j.  path[j] >= j, and places are left in
// ascending order, so each 16-byte column of the rows may be moved in place by
// one thread.  Bound by latency for few sequences (a dependent chain of lengths,
// tree, page table and rows: 5.5 us for one), and by HBM for many, which 128-byte
// rows from all over a large pool reach less of (3.6 TB/s).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace gpt2 {

namespace {

constexpr int kCtas = 8;  // per sequence, one cluster: its length is written when all of them have read it
constexpr int kThreads = 256;  // 64 sequences at 24 layers of 16 heads: 20.5 us; 128: 21.0, 512: 22.6, 1024: 30.6
constexpr int kBatch = 8;      // rows of a column on their way at a time (there: 4 the same, 16 25.6 us)

__global__ void __launch_bounds__(kThreads)
    draft_accept(uint4* __restrict__ pages, long long page_vecs, const int32_t* __restrict__ table, int32_t* lens,
                 const int32_t* __restrict__ refs, int T, const int32_t* __restrict__ tokens,
                 const int32_t* __restrict__ parents, const int32_t* __restrict__ counts,
                 const int32_t* __restrict__ chosen, int32_t* path, int32_t* n_kept, int32_t* next_tokens, int chunks,
                 int page_size, int max_pages, int n_pages, unsigned* err) {
  __shared__ int s_path[64];
  __shared__ int s_kept, s_last, s_moves;
  __shared__ long long s_from[64], s_to[64];  // of the rows that move: first vector of chunk 0
  griddep_wait();
  griddep_launch_dependents();
  const int rank = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int len = lens[b], n = counts ? min(counts[b], T) : T;
  if (tid < 32) {
    const int lane = tid;
    int kept = 0, last = 0, moves = 0;
    if (len >= 0 && n > 0 && len > max_pages * page_size - n) {
      if (lane == 0) record_error(err, kErrRange, kSitePagedLength);
      kept = -1;  // the sequence stays as it was
    } else if (len >= 0 && n > 0) {
      const long long at = static_cast<long long>(b) * T;
      int par[2], tok[2], cho[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = lane + 32 * e;
        par[e] = -2, tok[e] = cho[e] = 0;
        if (t < n) {
          par[e] = parents ? parents[at + t] : t - 1;
          tok[e] = tokens[at + t];
          cho[e] = chosen[at + t];
        }
      }
      int cur = 0;
      while (true) {
        if (lane == 0) s_path[kept] = cur;
        ++kept;
        const int c0 = __shfl_sync(0xffffffffu, cho[0], cur & 31), c1 = __shfl_sync(0xffffffffu, cho[1], cur & 31);
        last = cur < 32 ? c0 : c1;
        // a child stands behind its parent
        const unsigned m0 = __ballot_sync(0xffffffffu, lane > cur && par[0] == cur && tok[0] == last);
        const unsigned m1 = __ballot_sync(0xffffffffu, lane + 32 > cur && par[1] == cur && tok[1] == last);
        if ((m0 | m1) == 0) break;
        cur = m0 ? __ffs(static_cast<int>(m0)) - 1 : 31 + __ffs(static_cast<int>(m1));
      }
      __syncwarp();
      // where the rows stand; every place that is kept needs a page of its own
      const int32_t* row = table + static_cast<long long>(b) * max_pages;
      bool bad = false, shared = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = lane + 32 * e;
        long long from = 0, to = 0;
        bool move = false;
        if (j < kept) {
          const int p = s_path[j], a = (len + p) / page_size, z = (len + j) / page_size;
          const int from_page = row[a], to_page = row[z];
          if (from_page < 0 || from_page >= n_pages || to_page < 0 || to_page >= n_pages) {
            bad = true;
          } else {
            shared |= refs[to_page] > 1;
            from = from_page * page_vecs + (len + p - a * page_size) * 8;
            to = to_page * page_vecs + (len + j - z * page_size) * 8;
            move = p != j;
          }
        }
        const unsigned m = __ballot_sync(0xffffffffu, move);
        if (move) {
          const int k = moves + __popc(m & ((1u << lane) - 1));
          s_from[k] = from;
          s_to[k] = to;
        }
        moves += __popc(m);
      }
      bad = __any_sync(0xffffffffu, bad);
      shared = __any_sync(0xffffffffu, shared);
      if (bad || shared) {
        if (lane == 0) record_error(err, kErrRange, bad ? kSitePagedPage : kSitePagedShared);
        kept = -1;
        moves = 0;
      }
    }
    if (lane == 0) {
      s_kept = kept;
      s_last = last;
      s_moves = moves;
    }
  }
  // every CTA has the length: it may be written
  cluster_sync();
  __syncthreads();
  const int kept = s_kept, moves = s_moves;
  if (kept == 0) return;
  if (rank == 0) {
    if (kept < 0) {
      if (tid == 0) n_kept[b] = 0;
    } else {
      if (tid < T) path[static_cast<long long>(b) * T + tid] = tid < kept ? s_path[tid] : -1;
      if (tid == 0) {
        n_kept[b] = kept;
        next_tokens[b] = s_last;
        lens[b] = len + kept;
      }
    }
  }
  // a chunk: the K or V of one head of one layer, page_size rows of 8 vectors
  for (int i = rank * kThreads + tid; i < chunks * 8; i += kCtas * kThreads) {
    uint4* col = pages + static_cast<long long>(i >> 3) * page_size * 8 + (i & 7);
    for (int k0 = 0; k0 < moves; k0 += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < moves) x[k] = col[s_from[k0 + k]];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < moves) col[s_to[k0 + k]] = x[k];
    }
  }
}

// x[b T + t] = wte[token] + wpe[len + depth of t], one warp per row; zeros for
// rows behind n_draft, of idle slots, and (recorded) with a token or position
// out of range.
template <typename T16>
__global__ void __launch_bounds__(128)
    draft_embed(const int32_t* __restrict__ lens, int n_seq, int T, const int32_t* __restrict__ tokens,
                const int32_t* __restrict__ parents, const int32_t* __restrict__ counts,
                const T16* __restrict__ wte, const T16* __restrict__ wpe, float* __restrict__ x, int D, int V,
                int n_pos, unsigned* err) {
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= n_seq * T) return;
  const int b = row / T, t = row - b * T;
  const int len = lens[b], n = counts ? min(counts[b], T) : T;
  bool ok = len >= 0 && t < n;
  int tok = 0, pos = 0;
  if (ok) {
    int depth = t;
    if (parents) {
      const int32_t* up = parents + static_cast<long long>(b) * T;
      const int p0 = lane <= t ? up[lane] : -1, p1 = lane + 32 <= t ? up[lane + 32] : -1;
      int at = t;
      for (depth = 0; depth < t; ++depth) {
        const int q0 = __shfl_sync(0xffffffffu, p0, at & 31), q1 = __shfl_sync(0xffffffffu, p1, at & 31);
        const int p = at < 32 ? q0 : q1;
        if (p < 0 || p >= at) break;  // (the attention records a parent that is out of range)
        at = p;
      }
    }
    tok = tokens[row];
    const bool tok_ok = tok >= 0 && tok < V, pos_ok = len < n_pos && depth < n_pos - len;
    if (lane == 0 && !tok_ok) record_error(err, kErrRange, kSiteDecodeToken);
    if (lane == 0 && !pos_ok) record_error(err, kErrRange, kSiteDecodePos);
    ok = tok_ok && pos_ok;
    pos = len + depth;
  }
  const uint2* er = reinterpret_cast<const uint2*>(wte + static_cast<long long>(ok ? tok : 0) * D);
  const uint2* pr = reinterpret_cast<const uint2*>(wpe + static_cast<long long>(ok ? pos : 0) * D);
  float4* xr = reinterpret_cast<float4*>(x + static_cast<long long>(row) * D);
  for (int c = lane; c < D / 4; c += 32) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ok) {
      const uint2 e = er[c], p = pr[c];
      const float2 e0 = Type16<T16>::unpack2(e.x), e1 = Type16<T16>::unpack2(e.y);
      const float2 p0 = Type16<T16>::unpack2(p.x), p1 = Type16<T16>::unpack2(p.y);
      v = make_float4(e0.x + p0.x, e0.y + p0.y, e1.x + p1.x, e1.y + p1.y);
    }
    xr[c] = v;
  }
}

}  // namespace

cudaError_t launch_draft_embed(gpt2_dtype dt, const gpt2_paged_cache* c, int T, const int32_t* tokens,
                               const int32_t* parents, const int32_t* n_draft, const void* wte, const void* wpe,
                               float* x, int D, int V, int n_pos, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((c->n_seq * T + 3) / 4);
  if (dt == GPT2_F16)
    return launch_pdl(draft_embed<__half>, grid, 128, 0, s, 0, c->lens, c->n_seq, T, tokens, parents, n_draft,
                      static_cast<const __half*>(wte), static_cast<const __half*>(wpe), x, D, V, n_pos,
                      device_error_word());
  return launch_pdl(draft_embed<__nv_bfloat16>, grid, 128, 0, s, 0, c->lens, c->n_seq, T, tokens, parents, n_draft,
                    static_cast<const __nv_bfloat16*>(wte), static_cast<const __nv_bfloat16*>(wpe), x, D, V, n_pos,
                    device_error_word());
}

cudaError_t launch_draft_accept(const gpt2_paged_cache* c, int T, const int32_t* tokens, const int32_t* parents,
                                const int32_t* n_draft, const int32_t* chosen, int32_t* path, int32_t* n_kept,
                                int32_t* next_tokens, cudaStream_t s) {
  const int chunks = c->n_layer * 2 * c->n_kv_head;
  const long long page_vecs = static_cast<long long>(chunks) * c->page_size * 8;
  return launch_pdl(draft_accept, dim3(kCtas, c->n_seq), kThreads, 0, s, kCtas, static_cast<uint4*>(c->pages),
                    page_vecs, c->table, c->lens, c->refs, T, tokens, parents, n_draft, chosen, path, n_kept,
                    next_tokens, chunks, c->page_size, c->max_pages, c->n_pages, device_error_word());
}

}  // namespace gpt2
