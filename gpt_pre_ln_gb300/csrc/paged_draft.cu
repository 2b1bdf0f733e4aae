// Attention of up to 64 drafted tokens per sequence over a paged key-value
// cache (16-bit paths): the verification pass of speculative decoding.
//
//   out[b, t, h] = sum_{p visible to t} softmax_p(c q_th . k_p) v_p
//
// The drafted tokens of a sequence form a tree (parents[t] < t; -1 follows the
// cached positions).  They stand in the places len .. len + n - 1 behind the
// cached positions, token t stands for position len + depth(t), and it sees the
// cached positions, its ancestors and itself, all under the window's rule at
// its own position.  Query head h reads key-value head h / (n_head / n_kv_head).
//
// The n * (n_head / n_kv_head) query rows of one key-value head share its keys
// and values, which are read once for a block of up to 64 rows.  A position (256
// bytes) takes 4 * 64 flop a row: 64 rows are 64 flop a byte, a quarter of what
// the tensor cores need to be the limit.  The products are mma.sync m16n8k16 with
// 16 rows to a warp, whose scores and results stay in registers; with p as the sum
// of two 16-bit numbers they take 192 cycles of an SM's four tensor pipes for 64
// rows and 16 positions, which come from HBM in 170.  Up to 16 rows, the warps of a
// CTA take tiles of positions in turn, each from a ring of TMA boxes of its own;
// with more rows two or four warps share a ring, each with 16 rows of the block.
#include <algorithm>

#include "internal.h"
#include "paged.cuh"

namespace gpt2 {

namespace {

constexpr int kHd = 64;
constexpr int kTile = 16;  // positions per tile; page sizes are multiples of it
constexpr int kWarps = 4;  // warps per CTA; they take a piece's tiles in turn
constexpr int kThreads = kWarps * 32;
constexpr int kBoxBytes = kTile * kHd * 2;
constexpr int kTileBytes = 2 * kBoxBytes;  // K, then V
constexpr int kMinRun = 2 * kWarps;         // tiles per CTA at least
constexpr int kCtasPerSm = 4;

// WR: warps that share a ring, with 16 query rows each.  RIDE: up to 8 rows in
// all, whose other 8 carry the rounding remainder of p.
template <int WR, bool RIDE>
struct Shape {
  static constexpr int kRows = RIDE ? 8 : 16 * WR;
  static constexpr int kRings = kWarps / WR;
  static constexpr int kUnits = WR == 1 ? 1 : 2;       // tiles that a warp takes at a time
  static constexpr int kStages = WR == 1 ? 2 : 3 * WR / 2;  // of each ring: 128 or 192 KB of them on an SM
  static constexpr int kSlotBytes = kUnits * kTileBytes;
  static constexpr int kRingBytes = kStages * kSlotBytes;
};

template <typename T16>
struct DraftArgs {
  const T16* q;
  const T16* k;  // null: the drafted tokens' K and V are in the cache
  const T16* v;
  T16* out;
  float* lse;  // nullable, [n_seq * T, H]
  T16* pages;  // the layer's part of page 0
  int row0, page_rows;  // the pool as rows of 64: the layer's first row, rows per page
  const int32_t* table;
  const int32_t* lens;
  const int32_t* refs;
  const int32_t* parents;  // null: a chain
  const int32_t* counts;   // null: T each
  int* plan;        // base[n_seq + 1], then tiles per CTA
  float* part_o;    // [2 * CTAs, rows, 64]
  float2* part_ml;  // [2 * CTAs, rows]: running maximum (log2 units) and sum
  unsigned* err;
  long long ldq, ldkv, ldo;
  int n_pages, page_size, max_pages, n_seq, n_kv, H, group, T;
  int window, sinks;
  float scale_log2;  // score scale times log2(e)
};

// The tiles that some drafted token of a sequence sees: [0, ts) and
// [tw, tw + nt - ts), and its query rows per key-value head, in blocks.  nt < 0:
// nothing to do, the rows of the output are left alone.
struct Span {
  int len, n, ts, tw, nt, rows, blocks;
};
template <int ROWS, typename T16>
__device__ __forceinline__ Span span_of(const DraftArgs<T16>& a, int b, bool record) {
  Span s{0, 0, 0, 0, -1, 0, 0};
  const int len = a.lens[b], n = a.counts ? min(a.counts[b], a.T) : a.T;
  if (len < 0 || n <= 0) return s;
  if (len > a.max_pages * a.page_size - n) {
    if (record) record_error(a.err, kErrRange, kSitePagedLength);
    return s;
  }
  s.len = len;
  s.n = n;
  const int te = (len + n + kTile - 1) / kTile;
  if (a.window > 0 && len >= a.window) {
    const int first = len + 1 - a.window;  // of the tokens that follow the cached positions
    s.tw = first / kTile;
    s.ts = min((min(a.sinks, first) + kTile - 1) / kTile, s.tw);
  }
  s.nt = s.ts + te - s.tw;
  s.rows = n * a.group;
  s.blocks = (s.rows + ROWS - 1) / ROWS;
  return s;
}

// What the drafted tokens of one sequence see of one another (bit u of anc[t]),
// and how far behind the cached positions each stands.  One per warp.
struct Tree {
  unsigned long long anc[64];
  uint8_t depth[64];
};

template <typename T16>
__device__ __forceinline__ void build_tree(const DraftArgs<T16>& a, int b, const Span& sp, Tree& tree) {
  const int lane = threadIdx.x & 31;
  int up[2];  // the nearest ancestor that anc does not have yet
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = lane + 32 * e;
    up[e] = -1;
    if (t < sp.n) {
      int p = a.parents ? a.parents[static_cast<long long>(b) * a.T + t] : t - 1;
      if (p < -1 || p >= t) {
        record_error(a.err, kErrRange, kSiteDraftParent);
        p = -1;
      }
      up[e] = p;
    }
    tree.anc[t] = 1ull << t;
    tree.depth[t] = static_cast<uint8_t>(up[e]);
  }
  __syncwarp();
  // each round doubles the length of the path that anc holds
  for (int round = 0; round < 6; ++round) {
    if (!__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) break;
    unsigned long long more[2] = {0, 0};
    int far[2] = {-1, -1};
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (up[e] >= 0) {
        more[e] = tree.anc[up[e]];
        const int f = tree.depth[up[e]];
        far[e] = f == 255 ? -1 : f;
      }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      tree.anc[lane + 32 * e] |= more[e];
      up[e] = far[e];
      tree.depth[lane + 32 * e] = static_cast<uint8_t>(far[e]);
    }
    __syncwarp();
  }
  unsigned long long own[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    own[e] = tree.anc[lane + 32 * e];
    tree.depth[lane + 32 * e] = static_cast<uint8_t>(__popcll(own[e]) - 1);
  }
  __syncwarp();
  if (a.window > 0 && a.window < sp.n) {  // ancestors may be out of the window
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = tree.depth[lane + 32 * e];
      unsigned long long keep = 0;
      for (unsigned long long m = own[e]; m != 0; m &= m - 1) {
        const int u = __ffsll(static_cast<long long>(m)) - 1, du = tree.depth[u];
        if (d - du < a.window || sp.len + du < a.sinks) keep |= 1ull << u;
      }
      tree.anc[lane + 32 * e] = keep;
    }
    __syncwarp();
  }
}

// A ring of tiles.
struct Ring {
  const CUtensorMap* map;
  uint8_t* buf;     // [stages][K box, V box], 1024-byte aligned
  uint64_t* full;   // [stages]
  uint64_t* empty;  // [stages], where several warps share the ring
  int slot, parity;  // of the tile to take next
};

// What one warp makes of its tiles of one item: o (not divided by l), m (log2
// units) and l of its query rows.  Lane (r = lane / 4, j = lane % 4) holds rows r
// and r + 8: o[i] their dimensions 8i + 2j and 8i + 2j + 1.
struct Acc {
  float o[8][4];
  float m[2], l[2];
};

// One block of query rows of one key-value head of a sequence.
template <typename T16>
struct Item {
  Span sp;
  const int32_t* pages;  // the sequence's table row
  int b, kvh, block, row0, rows;  // its rows are row0 .. row0 + rows - 1 of the sequence's sp.rows
};

// Row i of an item: its token, and where its query head stands in q and out.
template <typename T16>
__device__ __forceinline__ void row_of(const DraftArgs<T16>& a, const Item<T16>& x, int i, int& t, int& head) {
  const int row = x.row0 + i;
  t = row / a.group;
  head = x.kvh * a.group + (row - t * a.group);
}
template <typename T16>
__device__ __forceinline__ const T16* q_row(const DraftArgs<T16>& a, const Item<T16>& x, int i) {
  int t, head;
  row_of(a, x, i, t, head);
  return a.q + (static_cast<long long>(x.b) * a.T + t) * a.ldq + static_cast<long long>(head) * kHd;
}

template <typename T16>
__device__ __forceinline__ uint32_t only_finite2(uint32_t w) {
  constexpr uint32_t kExp = std::is_same<T16, __half>::value ? 0x7c00u : 0x7f80u;
  if ((w & kExp) == kExp) w &= 0xffff0000u;
  if (((w >> 16) & kExp) == kExp) w &= 0xffffu;
  return w;
}

// p times a value that is not finite, of the first `places` places of the tile
// whose values are at vb: what the products with zero in their place have left out.
// (p below 0: not visible.)
template <typename T16, bool RIDE>
__device__ __forceinline__ void add_not_finite(Acc& acc, const float (&s)[2][4], const uint8_t* vb, int places) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
#pragma unroll 1
  for (int at = 0; at < places; ++at) {
    const int from = (r << 2) | ((at & 7) >> 1);
    float p[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float lo = (at & 1) ? s[0][2 * g + 1] : s[0][2 * g], hi = (at & 1) ? s[1][2 * g + 1] : s[1][2 * g];
      p[g] = __shfl_sync(0xffffffffu, at < 8 ? lo : hi, from);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(vb + at * 128 + ((i ^ (at & 7)) << 4) + 4 * j);
      if (w == only_finite2<T16>(w)) continue;
      const float2 v = Type16<T16>::unpack2(w);
#pragma unroll
      for (int g = 0; g < (RIDE ? 1 : 2); ++g) {
        if (p[g] < 0.f) continue;
        if (!isfinite(v.x)) acc.o[i][2 * g] += p[g] * v.x;
        if (!isfinite(v.y)) acc.o[i][2 * g + 1] += p[g] * v.y;
      }
    }
  }
}

// Four 8 x 8 tiles of 16-bit values, transposed; lane i gives the address of row
// i & 7 of tile i >> 3.
__device__ __forceinline__ void load_transposed(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
// The first product of a sum.
template <typename T16>
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T16, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Attention of query rows i0 .. i0 + 15 of an item over its tiles j0 .. j0 + cnt - 1 by
// one warp, kUnits of them at a time: those of ring `at`.  `leader`: the warp that
// fills the ring.  False if a wait ran out.
//
// The B fragments of q . k come out of shared memory as they are: sums over
// dimensions are free in their order, so lane (r, j) reads of key rows r and r + 8
// the dimensions 16j..16j+15 (q alike); those of p . v are read transposed.  With
// the boxes' 128-byte swizzle (16-byte unit u of row x at u ^ (x & 7)) no bank is
// read twice in a phase.
//
// Tiles with places behind the cached positions are brought by the lanes
// (16-byte asynchronous copies): cached places from their page, drafted ones
// from k and v, which are also stored in the page from here.
template <typename T16, int WR, bool RIDE>
__device__ __forceinline__ bool attend(const DraftArgs<T16>& a, const Item<T16>& x, int i0, bool leader, int at, int j0,
                                       int cnt, Ring& ring, Tree& tree, Acc& acc) {
  using S = Shape<WR, RIDE>;
  constexpr int kStages = S::kStages, U = S::kUnits;
  constexpr int kHalves = RIDE ? 1 : 2;  // row groups of a lane that hold rows
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int len = x.sp.len, end = len + x.sp.n;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc.o[i][e] = 0.f;
  acc.m[0] = acc.m[1] = -INFINITY;
  acc.l[0] = acc.l[1] = 0.f;
  const int units = (cnt + U - 1) / U, mine = units > at ? (units - at + S::kRings - 1) / S::kRings : 0;
  if (mine == 0) return true;
  // first position of tile u of this ring's i-th unit
  auto place = [&](int i, int u) {
    const int t = j0 + (at + i * S::kRings) * U + u;
    return (t < x.sp.ts ? t : x.sp.tw + (t - x.sp.ts)) * kTile;
  };
  auto there = [&](int i, int u) { return U == 1 || (at + i * S::kRings) * U + u < cnt; };
  // first row (K) of a tile in the pool, -1 when its page is not there (or there is no such tile); lane k of
  // tile k of the units from i on
  auto find_rows = [&](int i) {
    const int n = i + lane / U, u = lane % U;
    if (n >= mine || !there(n, u)) return -1;
    const int pos = place(n, u), c = pos / a.page_size;
    const int page = x.pages[c];
    if (page >= 0 && page < a.n_pages)
      return page * a.page_rows + a.row0 + x.kvh * a.page_size + (pos - c * a.page_size);
    record_error(a.err, kErrRange, kSitePagedPage);
    return -1;
  };
  int fetch32 = -1, rows32 = -1, fetched = 0;  // of the units to fetch, and of those to take
  auto issue = [&](int slot) {
    const int i = fetched++;
    if (i % (32 / U) == 0) fetch32 = find_rows(i);
    const uint32_t bar = smem_u32(&ring.full[slot]), base = smem_u32(ring.buf + slot * S::kSlotBytes);
    int boxes = 0, rows[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rows[u] = __shfl_sync(0xffffffffu, fetch32, (i * U + u) & 31);
      const uint32_t dst = base + u * kTileBytes;
      const int pos0 = place(i, u);
      if (rows[u] >= 0 && a.k && pos0 + kTile > len) {  // (the same for all lanes)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int y = (lane >> 3) + 4 * (k & 3), c = lane & 7, part = k >> 2, p = pos0 + y;
          const T16* from = nullptr;
          if (p < len)
            from = a.pages + (static_cast<long long>(rows[u] - a.row0) + y + part * a.n_kv * a.page_size) * kHd + c * 8;
          else if (p < end)
            from = (part ? a.v : a.k) + (static_cast<long long>(x.b) * a.T + (p - len)) * a.ldkv + x.kvh * kHd + c * 8;
          if (from)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + part * kBoxBytes + y * 128 +
                                                                           ((c ^ (y & 7)) << 4)),
                         "l"(from)
                         : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        rows[u] = -1;
      }
      boxes += rows[u] >= 0 ? 1 : 0;
    }
    __syncwarp();
    if (lane == 0) {
      if (boxes > 0)
        mbar_arrive_expect_tx(bar, boxes * kTileBytes);
      else
        mbar_arrive(bar);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (rows[u] >= 0) {
          tma_load_2d(base + u * kTileBytes, ring.map, bar, 0, rows[u]);
          tma_load_2d(base + u * kTileBytes + kBoxBytes, ring.map, bar, 0, rows[u] + a.n_kv * a.page_size);
        }
    }
  };
  if (leader) {
    int slot = ring.slot;
#pragma unroll 1
    for (int s = 0; s < kStages && fetched < mine; ++s) {
      issue(slot);
      slot = slot + 1 == kStages ? 0 : slot + 1;
    }
  }
  // q: lane (r, j) holds dimensions 16j..16j+15 of rows r and r + 8
  uint4 qf[4] = {};
#pragma unroll
  for (int g = 0; g < kHalves; ++g)
    if (i0 + 8 * g + r < x.rows) {
      const uint4* from = reinterpret_cast<const uint4*>(q_row(a, x, i0 + 8 * g + r) + 16 * j);
      qf[2 * g] = from[0];
      qf[2 * g + 1] = from[1];
    }
  const bool idle = i0 >= x.rows;  // no rows for this warp
  bool have_tree = false;
  // where this lane reads: of key rows r and r + 8, and of value row lane & 15
  const int k_at0 = r * 128 + (((2 * j) ^ r) << 4), k_at1 = r * 128 + (((2 * j + 1) ^ r) << 4);
  const int v_row = kBoxBytes + (lane & 15) * 128, v_unit = lane >> 4, v_swz = lane & 7;

  for (int i = 0; i < mine; ++i) {
    const bool ok = mbar_wait(smem_u32(&ring.full[ring.slot]), ring.parity);
    if (!__all_sync(0xffffffffu, ok)) {
      if (lane == 0) {
        record_error(a.err, kErrTimeout, kSitePagedLoad);
        for (int s = 0; s < kStages && i + s < mine; ++s) {  // the loads in flight must not outlive the CTA
          const int k = ring.slot + s;
          (void)mbar_wait(smem_u32(&ring.full[k % kStages]), ring.parity ^ (k >= kStages ? 1 : 0));
        }
      }
      __syncwarp();
      return false;
    }
    if (i % (32 / U) == 0) rows32 = find_rows(i);
    uint8_t* const tiles = ring.buf + ring.slot * S::kSlotBytes;
    int rows[U], pos0[U];
    bool any = false, whole = true;  // every row sees all of the tiles
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rows[u] = __shfl_sync(0xffffffffu, rows32, (i * U + u) & 31);
      pos0[u] = place(i, u);
      any |= rows[u] >= 0;
      whole = whole && rows[u] >= 0 && pos0[u] + kTile <= len &&
              (a.window <= 0 || pos0[u] >= end - a.window || pos0[u] + kTile <= a.sinks);
    }
    if (any && (!idle || leader)) {
      if (!whole) {
        if (!have_tree) {
          build_tree(a, x.b, x.sp, tree);
          have_tree = true;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // the drafted tokens' K and V into their page
          if (!leader || !a.k || x.block != 0 || rows[u] < 0 || pos0[u] + kTile <= len) continue;
          const int page = x.pages[pos0[u] / a.page_size];
          if (a.refs[page] > 1) {  // not into a page that other sequences read
            if (lane == 0) record_error(a.err, kErrRange, kSitePagedShared);
            continue;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int y = (lane >> 3) + 4 * (k & 3), c = lane & 7, part = k >> 2, p = pos0[u] + y;
            if (p >= len && p < end)
              *reinterpret_cast<uint4*>(
                  a.pages + (static_cast<long long>(rows[u] - a.row0) + y + part * a.n_kv * a.page_size) * kHd + c * 8) =
                  *reinterpret_cast<const uint4*>(tiles + u * kTileBytes + part * kBoxBytes + y * 128 +
                                                  ((c ^ (y & 7)) << 4));
          }
        }
      }
      float s[U][2][4];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint8_t* kr = tiles + u * kTileBytes + e * 1024;
          const uint4 k0 = *reinterpret_cast<const uint4*>(kr + k_at0);
          const uint4 k1 = *reinterpret_cast<const uint4*>(kr + k_at1);
          mma16816_first<T16>(s[u][e], qf[0].x, qf[2].x, qf[0].y, qf[2].y, k0.x, k0.y);
          mma16816<T16>(s[u][e], qf[0].z, qf[2].z, qf[0].w, qf[2].w, k0.z, k0.w);
          mma16816<T16>(s[u][e], qf[1].x, qf[3].x, qf[1].y, qf[3].y, k1.x, k1.y);
          mma16816<T16>(s[u][e], qf[1].z, qf[3].z, qf[1].w, qf[3].w, k1.z, k1.w);
        }
      uint32_t hidden = 0;  // bit 8u + 4e + 2g + k: score s[u][e][2g + k] is not visible
      if (!whole) {
#pragma unroll
        for (int g = 0; g < kHalves; ++g) {
          const int i_row = min(i0 + 8 * g + r, x.rows - 1);
          const int t = (x.row0 + i_row) / a.group;
          const unsigned long long anc = tree.anc[t];
          const int first = a.window > 0 ? len + tree.depth[t] + 1 - a.window : 0;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int p = pos0[u] + 8 * e + 2 * j + k;
                const bool seen = rows[u] >= 0 && (p < len ? (p >= first || p < a.sinks)
                                                           : p < end && ((anc >> (p - len)) & 1));
                if (!seen) {
                  s[u][e][2 * g + k] = -INFINITY;
                  hidden |= 1u << (8 * u + 4 * e + 2 * g + k);
                }
              }
        }
      }
      float alpha[2] = {1.f, 1.f};
#pragma unroll
      for (int g = 0; g < kHalves; ++g) {
        float mx = max3f(s[0][0][2 * g], s[0][0][2 * g + 1], s[0][1][2 * g]);
        if constexpr (U == 1)
          mx = fmaxf(mx, s[0][1][2 * g + 1]);
        else
          mx = max3f(max3f(mx, s[0][1][2 * g + 1], s[U - 1][0][2 * g]), s[U - 1][0][2 * g + 1],
                     fmaxf(s[U - 1][1][2 * g], s[U - 1][1][2 * g + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(acc.m[g], mx * a.scale_log2);
        const float ms = mn == -INFINITY ? 0.f : mn;  // every score so far is -inf
        alpha[g] = acc.m[g] == mn ? 1.f : ex2_approx(acc.m[g] - ms);
        acc.m[g] = mn;
        const float bias = kShift<T16> - ms;
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              s[u][e][2 * g + k] = ex2_approx(fmaf(s[u][e][2 * g + k], a.scale_log2, bias));
          sum += (s[u][0][2 * g] + s[u][0][2 * g + 1]) + (s[u][1][2 * g] + s[u][1][2 * g + 1]);
        }
        acc.l[g] = fmaf(acc.l[g], alpha[g], sum);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          acc.o[k][0] *= alpha[0];
          acc.o[k][1] *= alpha[0];
          acc.o[k][2] *= alpha[RIDE ? 0 : 1];
          acc.o[k][3] *= alpha[RIDE ? 0 : 1];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t vf[8][2];
        const uint32_t vb = smem_u32(tiles + u * kTileBytes) + v_row;
#pragma unroll
        for (int k = 0; k < 8; k += 2)
          load_transposed(vb + (((k + v_unit) ^ v_swz) << 4), vf[k][0], vf[k][1], vf[k + 1][0], vf[k + 1][1]);
        bool odd = false;  // a value that is not finite, in a tile that not every row sees all of
        if (!whole) {
          // places that nothing wrote may hold anything
          const int left = rows[u] >= 0 ? end - pos0[u] - 2 * j : 0;
          const uint32_t m0 = left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
          const uint32_t m1 = left >= 10 ? 0xffffffffu : left == 9 ? 0xffffu : 0u;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            vf[k][0] &= m0;
            vf[k][1] &= m1;
            const uint32_t f0 = only_finite2<T16>(vf[k][0]), f1 = only_finite2<T16>(vf[k][1]);
            odd |= f0 != vf[k][0] || f1 != vf[k][1];
            vf[k][0] = f0;
            vf[k][1] = f1;
          }
          odd = __any_sync(0xffffffffu, odd);
        }
        uint32_t ph[2][2], pl[2][2];  // [position half][row half]
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int g = 0; g < kHalves; ++g) split2<T16>(s[u][e][2 * g], s[u][e][2 * g + 1], ph[e][g], pl[e][g]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if constexpr (RIDE) {
            mma16816<T16>(acc.o[k], ph[0][0], pl[0][0], ph[1][0], pl[1][0], vf[k][0], vf[k][1]);
          } else {
            mma16816<T16>(acc.o[k], ph[0][0], ph[0][1], ph[1][0], ph[1][1], vf[k][0], vf[k][1]);
            mma16816<T16>(acc.o[k], pl[0][0], pl[0][1], pl[1][0], pl[1][1], vf[k][0], vf[k][1]);
          }
        }
        if (odd) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if ((hidden >> (8 * u + 4 * e + k)) & 1) s[u][e][k] = -1.f;
          add_not_finite<T16, RIDE>(acc, s[u], tiles + u * kTileBytes + kBoxBytes, min(kTile, end - pos0[u]));
        }
      }
    }
    // the slot is read: the unit kStages further on (where warps share the ring, into the slot before, which
    // the others have read by now)
    __syncwarp();
    if constexpr (WR == 1) {
      if (lane == 0) fence_proxy_async_smem();
      if (fetched < mine) issue(ring.slot);
    } else {
      if (lane == 0) mbar_arrive(smem_u32(&ring.empty[ring.slot]));
      if (leader && i > 0 && fetched < mine) {
        const int before = ring.slot == 0 ? kStages - 1 : ring.slot - 1;
        const bool free = mbar_wait(smem_u32(&ring.empty[before]), ring.slot == 0 ? ring.parity ^ 1 : ring.parity);
        if (!__all_sync(0xffffffffu, free)) {
          if (lane == 0) record_error(a.err, kErrTimeout, kSitePagedLoad);
          fetched = mine;  // (nothing more is brought: the waits for it run out)
        } else {
          issue(before);
        }
      }
    }
    if (++ring.slot == kStages) {
      ring.slot = 0;
      ring.parity ^= 1;
    }
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {  // sums over the four lanes of a row
    acc.l[g] += __shfl_xor_sync(0xffffffffu, acc.l[g], 1);
    acc.l[g] += __shfl_xor_sync(0xffffffffu, acc.l[g], 2);
  }
  if (RIDE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc.o[i][0] += acc.o[i][2];
      acc.o[i][1] += acc.o[i][3];
    }
  }
  return true;
}

// The rows of one warp's result: dst[row][64], ml[row] = (m, l).
template <typename T16, bool RIDE>
__device__ __forceinline__ void put_piece(const Acc& acc, int rows, float* dst, float2* ml) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
#pragma unroll
  for (int g = 0; g < (RIDE ? 1 : 2); ++g) {
    const int i = 8 * g + r;
    if (i >= rows) continue;
    float* po = dst + i * kHd + 2 * j;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<float2*>(po + 8 * k) = make_float2(acc.o[k][2 * g], acc.o[k][2 * g + 1]);
    if (j == 0) ml[i] = make_float2(acc.m[g] - kShift<T16>, acc.l[g]);
  }
}

// Four dimensions of row i of an item, and its log-sum-exp, into the output.
template <typename T16>
__device__ __forceinline__ void put_row(const DraftArgs<T16>& a, const Item<T16>& x, int i, int d4, const float4& acc,
                                        float M, float L) {
  int t, head;
  row_of(a, x, i, t, head);
  const long long token = static_cast<long long>(x.b) * a.T + t;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint2 v;
  v.x = Type16<T16>::pack2(acc.x * inv, acc.y * inv);
  v.y = Type16<T16>::pack2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(a.out + token * a.ldo + static_cast<long long>(head) * kHd + 4 * d4) = v;
  if (a.lse && d4 == 0) a.lse[token * a.H + head] = M + log2f(L);
}

// The rows of one warp's whole result into the output.
template <typename T16>
__device__ __forceinline__ void put_rows(const DraftArgs<T16>& a, const Item<T16>& x, int i0, const Acc& acc) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int i = i0 + 8 * g + r;
    if (i >= x.rows) continue;
    int t, head;
    row_of(a, x, i, t, head);
    const long long token = static_cast<long long>(x.b) * a.T + t;
    const float l = acc.l[g], inv = l == 0.f ? 0.f : 1.f / l;
    T16* to = a.out + token * a.ldo + static_cast<long long>(head) * kHd + 2 * j;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<uint32_t*>(to + 8 * k) =
          Type16<T16>::pack2(acc.o[k][2 * g] * inv, acc.o[k][2 * g + 1] * inv);
    if (a.lse && j == 0) a.lse[token * a.H + head] = acc.m[g] - kShift<T16> + log2f(l);
  }
}

template <typename T16>
__device__ __forceinline__ Item<T16> item_of(const DraftArgs<T16>& a, int b, int item, const Span& sp, int rows) {
  Item<T16> x;
  x.sp = sp;
  x.b = b;
  x.kvh = item / sp.blocks;
  x.block = item - x.kvh * sp.blocks;
  x.row0 = x.block * rows;
  x.rows = min(rows, sp.rows - x.row0);
  x.pages = a.table + static_cast<long long>(b) * a.max_pages;
  return x;
}

// Work is cut into equal runs of tiles over all (sequence, key-value head, row
// block) items laid end to end, one run per CTA, whatever the lengths are.  A CTA
// that holds all tiles of an item writes its output, pieces of an item go to the
// workspace and a second kernel joins them.  Rings of one or two warps take the
// tiles of a piece in turn and meet in shared memory.
template <typename T16, int WR, bool RIDE>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    draft_attn(const __grid_constant__ CUtensorMap map, const DraftArgs<T16> a) {
  using S = Shape<WR, RIDE>;
  constexpr int kRings = S::kRings;
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_bar[2][kRings * S::kStages];
  __shared__ int s_sum[kWarps];
  __shared__ float2 s_ml[kRings * S::kRows];
  __shared__ Tree s_tree[kWarps];
  uint8_t* s_tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  int* s_base = reinterpret_cast<int*>(s_tiles + kRings * S::kRingBytes);  // [n_seq + 1]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // which ring, and which 16 rows: not always the last ones on the same quarter of the SM
  const int at = warp / WR, rank = (warp + static_cast<int>(blockIdx.x)) % WR;
  const bool leader = rank == 0;
  Ring ring{&map, s_tiles + at * S::kRingBytes, s_bar[0] + at * S::kStages, s_bar[1] + at * S::kStages, 0, 0};
  if (tid == 0) {
    for (int s = 0; s < kRings * S::kStages; ++s) {
      mbar_init(smem_u32(&s_bar[0][s]), 1);
      mbar_init(smem_u32(&s_bar[1][s]), WR);
    }
    fence_barrier_init();
    tma_prefetch_desc(&map);
  }
  griddep_wait();
  // base[b] = tiles of all items of sequences before b
  int carry = 0;
  for (int b0 = 0; b0 < a.n_seq; b0 += kThreads) {
    const int b = b0 + tid;
    int v = 0;
    if (b < a.n_seq) {
      const Span sp = span_of<S::kRows>(a, b, blockIdx.x == 0);
      v = max(sp.nt, 0) * a.n_kv * sp.blocks;
    }
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
    if (b < a.n_seq) s_base[b] = before + incl - v;
    for (int w = 0; w < kWarps; ++w) carry += s_sum[w];
    __syncthreads();
  }
  if (tid == 0) s_base[a.n_seq] = carry;
  __syncthreads();
  const int total = carry;
  const int run = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), kMinRun);
  if (blockIdx.x == 0) {
    for (int b = tid; b <= a.n_seq; b += kThreads) a.plan[b] = s_base[b];
    if (tid == 0) a.plan[a.n_seq + 1] = run;
  }
  const long long t_first = static_cast<long long>(blockIdx.x) * run;
  if (t_first >= total) return;
  int t = static_cast<int>(t_first);
  const int t_end = static_cast<int>(min(t_first + run, static_cast<long long>(total)));

  while (t < t_end) {
    int lo = 0, hi = a.n_seq;  // last b with base[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_base[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const Span sp = span_of<S::kRows>(a, lo, false);
    const int item = (t - s_base[lo]) / sp.nt;
    const int j0 = (t - s_base[lo]) - item * sp.nt;  // first tile of this piece within the item
    const int cnt = min(sp.nt - j0, t_end - t);
    const Item<T16> x = item_of(a, lo, item, sp, S::kRows);
    const bool all = cnt == sp.nt;
    const long long part = 2ll * blockIdx.x + (t == static_cast<int>(t_first) ? 0 : 1);
    const int i0 = RIDE ? 0 : 16 * rank;
    Acc acc;
    const bool ok = attend<T16, WR, RIDE>(a, x, i0, leader, at, j0, cnt, ring, s_tree[warp], acc);
    t += cnt;
    __syncwarp();
    if constexpr (kRings == 1) {
      if (!ok) {
        // (the others' waits run out, too)
      } else if (all) {
        put_rows(a, x, i0, acc);
      } else {
        put_piece<T16, RIDE>(acc, x.rows - i0, a.part_o + (part * S::kRows + i0) * kHd, a.part_ml + part * S::kRows + i0);
      }
      if (t >= t_end) griddep_launch_dependents();
      fence_proxy_async_smem();
      if (!__syncthreads_and(ok)) return;  // (and every warp is through with the ring)
    } else {
      // a warp's result (fp32 rows of 64) takes the place of its ring
      if (WR > 1 && !__syncthreads_and(ok)) return;
      const int pieces = min((cnt + S::kUnits - 1) / S::kUnits, kRings);
      if (at < pieces && ok)
        put_piece<T16, RIDE>(acc, x.rows - i0, reinterpret_cast<float*>(ring.buf) + i0 * kHd, s_ml + at * S::kRows + i0);
      if (!__syncthreads_and(ok)) return;
      if (t >= t_end) griddep_launch_dependents();
      for (int k = tid; k < x.rows * 16; k += kThreads) {
        const int i = k >> 4, d4 = k & 15;
        float M = -INFINITY, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < pieces; ++w)
          merge(o, M, L, *reinterpret_cast<const float4*>(s_tiles + w * S::kRingBytes + (i * kHd + 4 * d4) * 4),
                s_ml[w * S::kRows + i]);
        if (all) {
          put_row(a, x, i, d4, o, M, L);
        } else {
          *reinterpret_cast<float4*>(a.part_o + (part * S::kRows + i) * kHd + 4 * d4) = o;
          if (d4 == 0) a.part_ml[part * S::kRows + i] = make_float2(M, L);
        }
      }
      // the rings take tiles again: generic accesses before asynchronous writes
      fence_proxy_async_smem();
      __syncthreads();
    }
  }
}

// Joins the pieces of items that several CTAs shared, in a fixed order.  One
// CTA for `width` rows of an item, side by side, 16 threads for a row's 64
// dimensions; the threads that are left take every ways-th piece.
constexpr int kJoinThreads = 256;
template <typename T16, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) draft_join(const DraftArgs<T16> a, int width, int max_blocks) {
  __shared__ float4 s_o[kJoinThreads];
  __shared__ float2 s_ml[kJoinThreads];
  const int per_seq = a.n_kv * max_blocks;
  const int b = blockIdx.x / per_seq, item = blockIdx.x - b * per_seq;
  // the lengths are older than the kernel before, which has waited for them
  const Span sp = span_of<ROWS>(a, b, false);
  griddep_wait();
  griddep_launch_dependents();
  if (sp.nt < 0 || item >= a.n_kv * sp.blocks) return;
  const Item<T16> x = item_of(a, b, item, sp, ROWS);
  const int first_row = blockIdx.y * width;
  if (first_row >= x.rows) return;
  const int run = a.plan[a.n_seq + 1];
  const int start = a.plan[b] + item * sp.nt;
  const int w0 = start / run, w1 = (start + sp.nt - 1) / run;
  if (w0 == w1) return;  // that CTA wrote the output
  const bool second = start != w0 * run;  // the item began within the first CTA's run: its second piece
  const int ways = kJoinThreads / 16 / width;
  const int tid = threadIdx.x, d4 = tid & 15, way = (tid >> 4) / width;
  const int i = first_row + (tid >> 4) % width;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < x.rows) {
    constexpr int kAhead = 4;  // pieces on their way at a time
    for (int w = w0 + way; w <= w1; w += kAhead * ways) {
      float4 o[kAhead];
      float2 ml[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int wu = w + u * ways;
        ml[u] = make_float2(-INFINITY, 0.f);
        if (wu <= w1) {
          const long long at = (2ll * wu + (wu == w0 && second ? 1 : 0)) * ROWS + i;
          ml[u] = a.part_ml[at];
          o[u] = *reinterpret_cast<const float4*>(a.part_o + at * kHd + 4 * d4);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) merge(acc, M, L, o[u], ml[u]);
    }
  }
  // pairwise, in an order that the number of threads alone gives
  s_o[tid] = acc;
  s_ml[tid] = make_float2(M, L);
  for (int k = ways >> 1; k > 0; k >>= 1) {
    __syncthreads();
    if (way < k) {
      merge(acc, M, L, s_o[tid + 16 * width * k], s_ml[tid + 16 * width * k]);
      s_o[tid] = acc;
      s_ml[tid] = make_float2(M, L);
    }
  }
  if (way == 0 && i < x.rows) put_row(a, x, i, d4, acc, M, L);
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Query rows per block for T tokens of a group of heads: few rows leave the warps
// their own tiles (and, up to 8, carry the remainder of p for nothing), more of
// them read the cache less often.
int rows_of(int T, int group) {
  const int rows = T * group;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

template <typename T16, int WR, bool RIDE>
cudaError_t launch_kind(const CUtensorMap& map, const DraftArgs<T16>& a, cudaStream_t s) {
  using S = Shape<WR, RIDE>;
  constexpr int kFixed = S::kRings * S::kRingBytes + 1024;
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(draft_attn<T16, WR, RIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kFixed + (kMaxPagedSeqs + 1) * 4);
    if (e != cudaSuccess) return e;
    // the join leaves the SMs split as draft_attn has them: between two splits an SM has to run empty
    e = cudaFuncSetAttribute(draft_join<T16, S::kRows>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  const int sms = num_sms();
  cudaError_t e = launch_pdl(draft_attn<T16, WR, RIDE>, sms * kCtasPerSm, kThreads, kFixed + (a.n_seq + 1) * 4, s, 0,
                             map, a);
  if (e != cudaSuccess) return e;
  const int max_blocks = (a.T * a.group + S::kRows - 1) / S::kRows;
  const long long items = static_cast<long long>(a.n_seq) * a.n_kv * max_blocks;
  const int most = std::min(S::kRows, a.T * a.group);
  int width = 1;  // as many CTAs as there are places for
  while (width < 16 && items * ((most + width - 1) / width) > 4 * sms) width *= 2;
  return launch_pdl(draft_join<T16, S::kRows>, dim3(static_cast<unsigned>(items), (most + width - 1) / width),
                    kJoinThreads, 0, s, 0, a, width, max_blocks);
}

template <typename T16>
cudaError_t launch_t(const gpt2_paged_cache* c, int layer, const void* q, int64_t ldq, const void* k, const void* v,
                     int64_t ldkv, void* out, int64_t ldo, float* lse, int T, const int32_t* parents,
                     const int32_t* n_draft, int n_head, float score_scale, int window, int sinks, void* ws,
                     cudaStream_t s) {
  DraftArgs<T16> a;
  a.q = static_cast<const T16*>(q);
  a.k = static_cast<const T16*>(k);
  a.v = static_cast<const T16*>(v);
  a.out = static_cast<T16*>(out);
  a.lse = lse;
  const long long layer_elems = 2ll * c->n_kv_head * c->page_size * kHd;
  a.pages = static_cast<T16*>(c->pages) + layer * layer_elems;
  a.page_rows = c->n_layer * 2 * c->n_kv_head * c->page_size;
  a.row0 = layer * 2 * c->n_kv_head * c->page_size;
  a.table = c->table;
  a.lens = c->lens;
  a.refs = c->refs;
  a.parents = parents;
  a.counts = n_draft;
  a.err = device_error_word();
  a.ldq = ldq;
  a.ldkv = ldkv;
  a.ldo = ldo;
  a.n_pages = c->n_pages;
  a.page_size = c->page_size;
  a.max_pages = c->max_pages;
  a.n_seq = c->n_seq;
  a.n_kv = c->n_kv_head;
  a.H = n_head;
  a.group = n_head / c->n_kv_head;
  a.T = T;
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = score_scale * 1.4426950408889634f;
  const int rows = rows_of(T, a.group);
  const size_t slots = 2ull * num_sms() * kCtasPerSm * rows;
  char* base = static_cast<char*>(ws);
  a.plan = reinterpret_cast<int*>(base);
  base += align256((static_cast<size_t>(c->n_seq) + 2) * 4);
  a.part_ml = reinterpret_cast<float2*>(base);
  base += align256(slots * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(base);
  // the pool as one [rows, 64] matrix
  CUtensorMap map;
  if (!encode_tma_2d(&map, Type16<T16>::kTma, c->pages, kHd, static_cast<uint64_t>(c->n_pages) * a.page_rows, kHd * 2,
                     kHd, kTile))
    return cudaErrorInvalidValue;
  switch (rows) {
    case 8: return launch_kind<T16, 1, true>(map, a, s);
    case 16: return launch_kind<T16, 1, false>(map, a, s);
    case 32: return launch_kind<T16, 2, false>(map, a, s);
    default: return launch_kind<T16, 4, false>(map, a, s);
  }
}

}  // namespace

size_t attention_draft_workspace(const gpt2_paged_cache* c, int T, int n_head) {
  const size_t slots = 2ull * num_sms() * kCtasPerSm * rows_of(T, n_head / c->n_kv_head);
  return align256((static_cast<size_t>(c->n_seq) + 2) * 4) + align256(slots * sizeof(float2)) +
         align256(slots * kHd * 4);
}

bool attention_draft_fits(const gpt2_paged_cache* c, int T, int n_head) {
  // rows of the pool are TMA coordinates, and tiles of all items are counted, in
  // 32 bits, the latter with room for one run more
  if (static_cast<double>(c->n_pages) * c->n_layer * 2 * c->n_kv_head * c->page_size >= 2147483648.0) return false;
  const int rows = rows_of(T, n_head / c->n_kv_head);
  const long long blocks = (static_cast<long long>(T) * (n_head / c->n_kv_head) + rows - 1) / rows;
  return static_cast<long long>(c->n_seq) * c->n_kv_head * blocks *
             (static_cast<long long>(c->max_pages) * c->page_size / kTile) <
         (1ll << 30);
}

cudaError_t launch_attention_draft(const gpt2_paged_cache* c, int layer, const void* q, int64_t ldq, const void* k,
                                   const void* v, int64_t ldkv, void* out, int64_t ldo, float* lse, int T,
                                   const int32_t* parents, const int32_t* n_draft, int n_head, float score_scale,
                                   int window, int sinks, void* ws, cudaStream_t s) {
  return c->dtype == GPT2_F16 ? launch_t<__half>(c, layer, q, ldq, k, v, ldkv, out, ldo, lse, T, parents, n_draft,
                                                 n_head, score_scale, window, sinks, ws, s)
                              : launch_t<__nv_bfloat16>(c, layer, q, ldq, k, v, ldkv, out, ldo, lse, T, parents,
                                                        n_draft, n_head, score_scale, window, sinks, ws, s);
}

}  // namespace gpt2
