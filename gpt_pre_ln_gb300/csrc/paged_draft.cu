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
// rows and 16 positions, which come from HBM in 170.
//
// Up to 16 rows, the warps of a CTA take tiles of 16 positions in turn, each from a
// ring of TMA boxes that it fills itself.  With more rows two or four warps take the
// same tiles, 32 positions at a time, each with 16 rows of the block, and a fifth
// warp brings them: the warp that also filled the ring held up all four (64 rows,
// 16 sequences of 4096: 116 us, with the fifth warp 82; 48 rows, 8 of 32768: 109 and
// 80).  Up to 16 rows the fifth warp cost more than it gave (16 rows, 32 sequences
// of up to 1087: 28 us without, 39 with it).
//
// What bounds it with many rows is how fast one warp gets through the instructions
// around the products (exponentials, the split of p, running maxima: 400 for 16 rows
// and 32 positions at 4 cycles each), not memory and not the products: 2.4 TB/s and
// 39% of the tensor pipes at 64 rows; with 7 rows it is memory (5.1 TB/s).
#include <algorithm>

#include "internal.h"
#include "paged.cuh"

namespace gpt2 {

namespace {

constexpr int kHd = 64;
constexpr int kTile = 16;  // positions per tile; page sizes are multiples of it
constexpr int kWarps = 4;  // warps per CTA that take tiles
constexpr int kTakers = kWarps * 32;
constexpr int kBoxBytes = kTile * kHd * 2;
constexpr int kTileBytes = 2 * kBoxBytes;  // K, then V
constexpr int kMinRun = 2 * kWarps;        // tiles per CTA at least

// WR: warps that take the same tiles, with 16 query rows each.  RIDE: up to 8 rows
// in all, whose other 8 carry the rounding remainder of p.
template <int WR, bool RIDE>
struct Shape {
  static constexpr int kRows = RIDE ? 8 : 16 * WR;
  static constexpr int kGroups = kWarps / WR;
  static constexpr bool kBringer = WR > 1;          // a warp that brings the tiles
  static constexpr int kUnit = kBringer ? 2 : 1;    // tiles that a warp takes at a time
  static constexpr int kRings = kBringer ? 1 : kWarps;
  static constexpr int kSlots = kBringer ? 6 : 2;   // units in a ring: 144 or 128 KB of them on an SM
  static constexpr int kCtas = kBringer ? 3 : 4;    // per SM
  static constexpr int kThreads = kTakers + (kBringer ? 32 : 0);
  static constexpr int kRingBytes = kSlots * kUnit * kTileBytes;
  // where the groups' results (fp32 rows of 64) meet: their rings, or a place of its own
  static constexpr int kMeetBytes = kBringer && kGroups > 1 ? kGroups * kRows * kHd * 4 : 0;
  // A slot's uses one after another belong to one group: a wait for the phase after the next would not wait.
  static_assert(!kBringer || kSlots % kGroups == 0, "slots are a multiple of the groups");
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
  int n_layer, layer;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* refs;
  const int32_t* parents;  // null: a chain
  const int32_t* counts;   // null: T each
  int* plan;        // base[n_seq + 1], then tiles per CTA (below 0: items are rounded up to whole runs)
  float* part_o;    // [2 * CTAs, rows, 64]
  float2* part_ml;  // [2 * CTAs, rows]: running maximum (log2 units) and sum
  unsigned* err;
  long long ldq, ldkv, ldo;
  int n_pages, page_size, max_pages, n_seq, n_kv, H, group, T;
  int window, sinks;
  int items;  // at most
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
  int odd;  // values that are not finite have been left out of the products
};

// The paths up to the cached positions.
template <typename T16>
__device__ __forceinline__ void find_ancestors(const DraftArgs<T16>& a, int b, const Span& sp, Tree& tree) {
  const int lane = threadIdx.x & 31;
  int up[2];  // the nearest ancestor that anc does not have yet
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = lane + 32 * e;
    up[e] = -1;
    if (t < sp.n) {
      int p = a.parents[static_cast<long long>(b) * a.T + t];
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
#pragma unroll
  for (int e = 0; e < 2; ++e)
    tree.depth[lane + 32 * e] = static_cast<uint8_t>(__popcll(tree.anc[lane + 32 * e]) - 1);
  __syncwarp();
}

template <typename T16>
__device__ __forceinline__ void build_tree(const DraftArgs<T16>& a, int b, const Span& sp, Tree& tree) {
  const int lane = threadIdx.x & 31;
  if (!a.parents) {  // a chain
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      tree.anc[lane + 32 * e] = ~0ull >> (63 - lane - 32 * e);
      tree.depth[lane + 32 * e] = static_cast<uint8_t>(lane + 32 * e);
    }
    __syncwarp();
  } else {
    find_ancestors(a, b, sp, tree);
  }
  if (a.window > 0 && a.window < sp.n) {  // ancestors may be out of the window
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = tree.depth[lane + 32 * e];
      unsigned long long keep = 0;
      for (unsigned long long m = tree.anc[lane + 32 * e]; m != 0; m &= m - 1) {
        const int u = __ffsll(static_cast<long long>(m)) - 1, du = tree.depth[u];
        if (d - du < a.window || sp.len + du < a.sinks) keep |= 1ull << u;
      }
      tree.anc[lane + 32 * e] = keep;
    }
    __syncwarp();
  }
}

// A unit of tiles in the ring: their first rows (K) in the pool, -1 where there is
// no such tile or its page is not there, and positions; pos[0] < 0: every query row
// sees all of them.
template <int U>
struct Unit {
  int row[U], pos[U];
};
template <int U>
struct Ring {
  uint8_t* buf;     // [slots][U][K box, V box], 1024-byte aligned
  Unit<U>* unit;    // [slots]
  uint64_t* full;   // [slots]
  uint64_t* empty;  // [slots]
};
// Where a warp is in a ring.
template <int SLOTS>
struct Turn {
  int slot, parity;
  __device__ __forceinline__ void step(int n) {  // at most SLOTS
    slot += n;
    if (slot >= SLOTS) {
      slot -= SLOTS;
      parity ^= 1;
    }
  }
  __device__ __forceinline__ void advance(int n) {
    parity ^= ((slot + n) / SLOTS) & 1;
    slot = (slot + n) % SLOTS;
  }
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

// Brings one unit of tiles into a slot of the ring (a whole warp).
//
// Tiles with places behind the cached positions are brought by the lanes
// (16-byte asynchronous copies): cached places from their page, drafted ones
// from k and v.  True if there were any.
template <typename T16, int U>
__device__ __forceinline__ bool bring(const CUtensorMap* map, const DraftArgs<T16>& a, const Item<T16>& x, Unit<U> unit,
                                      const int (&page)[U], const Ring<U>& ring, int slot) {
  const int lane = threadIdx.x & 31, len = x.sp.len, end = len + x.sp.n;
  bool whole = true, by_lanes = false;
  int boxes = 0, tma[U];
  const uint32_t bar = smem_u32(&ring.full[slot]), base = smem_u32(ring.buf + slot * U * kTileBytes);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = unit.row[u], pos0 = unit.pos[u];
    tma[u] = at;
    whole = whole && at >= 0 && pos0 + kTile <= len &&
            (a.window <= 0 || pos0 >= end - a.window || pos0 + kTile <= a.sinks);
    if (at >= 0 && a.k && pos0 + kTile > len) {  // (the same for all lanes)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int y = (lane >> 3) + 4 * (k & 3), c = lane & 7, part = k >> 2, p = pos0 + y;
        const T16* from = nullptr;
        if (p < len)
          from = a.pages + (static_cast<long long>(at - a.row0) + y + part * a.n_kv * a.page_size) * kHd + c * 8;
        else if (p < end)
          from = (part ? a.v : a.k) + (static_cast<long long>(x.b) * a.T + (p - len)) * a.ldkv + x.kvh * kHd + c * 8;
        if (from)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + u * kTileBytes + part * kBoxBytes +
                                                                         y * 128 + ((c ^ (y & 7)) << 4)),
                       "l"(from)
                       : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
      tma[u] = -1;
      by_lanes = true;
    }
    boxes += tma[u] >= 0 ? 1 : 0;
  }
  __syncwarp();
  if (lane == 0) {
    if (whole) unit.pos[0] = -1;
    ring.unit[slot] = unit;
    if (boxes > 0)
      mbar_arrive_expect_tx(bar, boxes * kTileBytes);
    else
      mbar_arrive(bar);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (tma[u] >= 0)  // K and V
        tma_load_4d(base + u * kTileBytes, map, bar, 0, tma[u] - page[u] * a.page_rows - a.row0, 0,
                    page[u] * a.n_layer + a.layer);
  }
  __syncwarp();
  return by_lanes;
}

// First positions, rows and pages of tiles j0, j0 + step, ... of an item, 32 at a time: those
// of tile i + lane of them.
template <typename T16>
__device__ __forceinline__ void find_tiles(const DraftArgs<T16>& a, const Item<T16>& x, int j0, int step, int i, int cnt,
                                           int& row, int& pos, int& page) {
  const int n = i + static_cast<int>(threadIdx.x & 31), t = j0 + n * step;
  row = -1;
  page = 0;
  pos = (t < x.sp.ts ? t : x.sp.tw + (t - x.sp.ts)) * kTile;
  if (n >= cnt) return;
  const int c = pos / a.page_size;
  page = x.pages[c];
  if (page >= 0 && page < a.n_pages)
    row = page * a.page_rows + a.row0 + x.kvh * a.page_size + (pos - c * a.page_size);
  else
    record_error(a.err, kErrRange, kSitePagedPage);
}

// The warp that brings tiles j0 .. j0 + cnt - 1 of an item; by_lanes: a bit for each slot that lanes wrote last.
// False if a wait ran out.
template <typename T16, int U, int SLOTS>
__device__ __forceinline__ bool bring_all(const CUtensorMap* map, const DraftArgs<T16>& a, const Item<T16>& x, int j0,
                                          int cnt, const Ring<U>& ring, Turn<SLOTS>& turn, bool& around,
                                          unsigned& by_lanes) {
  int row = -1, pos = 0, page = 0;
  for (int i = 0; i < cnt; i += U) {
    if ((i & 31) == 0) find_tiles(a, x, j0, 1, i, cnt, row, pos, page);
    if (around) {
      const bool free = mbar_wait(smem_u32(&ring.empty[turn.slot]), turn.parity ^ 1);
      if (!__all_sync(0xffffffffu, free)) {
        if ((threadIdx.x & 31) == 0) record_error(a.err, kErrTimeout, kSitePagedLoad);
        return false;
      }
      // what the lanes wrote there, before the asynchronous writes that may follow
      if ((by_lanes >> turn.slot) & 1) fence_proxy_async_smem();
    }
    Unit<U> unit;
    int of[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      of[u] = __shfl_sync(0xffffffffu, page, (i + u) & 31);
      unit.row[u] = __shfl_sync(0xffffffffu, row, (i + u) & 31);
      unit.pos[u] = __shfl_sync(0xffffffffu, pos, (i + u) & 31);
    }
    const unsigned bit = 1u << turn.slot;
    by_lanes = bring<T16, U>(map, a, x, unit, of, ring, turn.slot) ? by_lanes | bit : by_lanes & ~bit;
    turn.step(1);
    if (turn.slot == 0) around = true;
  }
  return true;
}

// 16 query rows from i0 on, as the A operands of q . k.
struct Query {
  uint32_t a[4][4];
};

// One unit of tiles by one warp; MASKED: not every row sees all of it, and values that
// are not finite are left out.
//
// The B fragments of q . k come out of shared memory as they are: sums over
// dimensions are free in their order, so lane (r, j) reads of key rows r and r + 8
// the dimensions 16j..16j+15 (q alike); those of p . v are read transposed.  With
// the boxes' 128-byte swizzle (16-byte unit u of row x at u ^ (x & 7)) no bank is
// read twice in a phase.
template <typename T16, bool RIDE, bool MASKED, int U>
__device__ __forceinline__ void take(const DraftArgs<T16>& a, const Item<T16>& x, int i0, const Query& q,
                                     const uint8_t* tiles, const Unit<U>& unit, Tree& tree, Acc& acc) {
  constexpr int kHalves = RIDE ? 1 : 2;  // row groups of a lane that hold rows
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int len = x.sp.len, end = len + x.sp.n;
  float s[U][2][4];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint8_t* kr = tiles + u * kTileBytes + (r + 8 * e) * 128;
      const uint4 k0 = *reinterpret_cast<const uint4*>(kr + (((2 * j) ^ r) << 4));
      const uint4 k1 = *reinterpret_cast<const uint4*>(kr + (((2 * j + 1) ^ r) << 4));
      mma16816_first<T16>(s[u][e], q.a[0][0], q.a[0][1], q.a[0][2], q.a[0][3], k0.x, k0.y);
      mma16816<T16>(s[u][e], q.a[1][0], q.a[1][1], q.a[1][2], q.a[1][3], k0.z, k0.w);
      mma16816<T16>(s[u][e], q.a[2][0], q.a[2][1], q.a[2][2], q.a[2][3], k1.x, k1.y);
      mma16816<T16>(s[u][e], q.a[3][0], q.a[3][1], q.a[3][2], q.a[3][3], k1.z, k1.w);
    }
  if constexpr (MASKED) {
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
            const int p = unit.pos[u] + 8 * e + 2 * j + k;
            const bool seen = unit.row[u] >= 0 && (p < len ? (p >= first || p < a.sinks)
                                                           : p < end && ((anc >> (p - len)) & 1));
            if (!seen) s[u][e][2 * g + k] = -INFINITY;
          }
    }
  }
  float alpha[2] = {1.f, 1.f};
#pragma unroll
  for (int g = 0; g < kHalves; ++g) {
    float mx = max3f(s[0][0][2 * g], s[0][0][2 * g + 1], fmaxf(s[0][1][2 * g], s[0][1][2 * g + 1]));
#pragma unroll
    for (int u = 1; u < U; ++u)
      mx = max3f(max3f(mx, s[u][0][2 * g], s[u][0][2 * g + 1]), s[u][1][2 * g], s[u][1][2 * g + 1]);
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
        for (int k = 0; k < 2; ++k) s[u][e][2 * g + k] = ex2_approx(fmaf(s[u][e][2 * g + k], a.scale_log2, bias));
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
  const uint32_t v_row = smem_u32(tiles) + kBoxBytes + (lane & 15) * 128;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t vf[8][2];
#pragma unroll
    for (int k = 0; k < 8; k += 2)
      load_transposed(v_row + u * kTileBytes + (((k + (lane >> 4)) ^ (lane & 7)) << 4), vf[k][0], vf[k][1], vf[k + 1][0],
                      vf[k + 1][1]);
    if constexpr (MASKED) {
      bool odd = false;
      // places that nothing wrote may hold anything
      const int left = unit.row[u] >= 0 ? end - unit.pos[u] - 2 * j : 0;
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
      if (odd) tree.odd = 1;
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
  }
}

// The drafted tokens' K and V of a unit from shared memory into their pages.
template <typename T16, int U>
__device__ __forceinline__ void store_drafts(const DraftArgs<T16>& a, const Item<T16>& x, const uint8_t* tiles,
                                             const Unit<U>& unit) {
  const int lane = threadIdx.x & 31, len = x.sp.len, end = len + x.sp.n;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (unit.row[u] < 0 || unit.pos[u] + kTile <= len) continue;
    const int page = x.pages[unit.pos[u] / a.page_size];
    if (a.refs[page] > 1) {  // not into a page that other sequences read
      if (lane == 0) record_error(a.err, kErrRange, kSitePagedShared);
      continue;
    }
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      const int y = (lane >> 3) + 4 * (k & 3), c = lane & 7, part = k >> 2, p = unit.pos[u] + y;
      if (p >= len && p < end)
        *reinterpret_cast<uint4*>(
            a.pages + (static_cast<long long>(unit.row[u] - a.row0) + y + part * a.n_kv * a.page_size) * kHd + c * 8) =
            *reinterpret_cast<const uint4*>(tiles + u * kTileBytes + part * kBoxBytes + y * 128 + ((c ^ (y & 7)) << 4));
    }
  }
}

// What the values that are not finite make of the results of query rows i0 .. i0 + 15
// of an item, over units at, at + step, ... (of U tiles) of tiles j0 .. j0 + cnt - 1.
// p v is infinite wherever p is above 0, however small, and NaN with p = 0 (a score of
// -inf) or beside the other infinity, wherever the value stands.  The products
// would have it by the tile: with p in two parts 0 * inf or a negative remainder makes
// NaN of inf, and where rows differ in what they see they cannot have it at all.
//
// Bit 4k + 2g + e of a lane (r, j), for dimension 8k + 2j + e of row r + 8g: +inf or NaN
// in the low half, -inf or NaN in the high one.  From global memory, a tile's values at
// once (1 us); a place that has such values is looked at for itself, and its score where
// they decide something.  16 sequences of 4096, 64 tokens each: 84 us, 187 with one
// infinity in one of them, 314 with one in each page, 1000 with nothing but NaN, 3100
// with nothing but infinities.
template <typename T16, int U>
__device__ __noinline__ unsigned long long not_finite(const DraftArgs<T16>& a, const Item<T16>& x, int i0, int at,
                                                      int step, int j0, int cnt, const Tree& tree) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int len = x.sp.len, end = len + x.sp.n;
  unsigned up = 0, down = 0;
#pragma unroll 1
  for (int n = at * U; n < cnt; n += (n + 1) % U ? 1 : 1 + (step - 1) * U) {
    const int tile = j0 + n, pos = (tile < x.sp.ts ? tile : x.sp.tw + (tile - x.sp.ts)) * kTile, c = pos / a.page_size;
    const int page = x.pages[c];
    if (page < 0 || page >= a.n_pages) continue;
    const int places = min(kTile, end - pos);
    // K and V of the tile's first place, in the cache and (drafted places) where they are brought from
    const T16* ck =
        a.pages + (static_cast<long long>(page) * a.page_rows + x.kvh * a.page_size + (pos - c * a.page_size)) * kHd;
    const T16* cv = ck + static_cast<long long>(a.n_kv) * a.page_size * kHd;
    const long long ld = a.k ? a.ldkv : kHd, first = (static_cast<long long>(x.b) * a.T + (pos - len)) * ld + x.kvh * kHd;
    const T16 *dk = a.k ? a.k + first : ck, *dv = a.k ? a.v + first : cv;
    uint32_t w[kTile];  // (no load waits for a branch or for another: one after another they take ten times as long)
#pragma unroll
    for (int y = 0; y < kTile; ++y) {
      const int z = min(y, places - 1);
      const T16* v = pos + z >= len ? dv + z * ld : cv + z * kHd;
      w[y] = reinterpret_cast<const uint32_t*>(v)[lane];
    }
    unsigned odd = 0;  // bit y: place y has some
#pragma unroll
    for (int y = 0; y < kTile; ++y) odd |= w[y] != only_finite2<T16>(w[y]) ? 1u << y : 0u;
    odd = __reduce_or_sync(0xffffffffu, odd) & ((1u << places) - 1);
#pragma unroll 1
    for (; odd != 0; odd &= odd - 1) {
      const int y = __ffs(static_cast<int>(odd)) - 1, p = pos + y;
      const T16 *k_row = p >= len ? dk + y * ld : ck + y * kHd, *v_row = p >= len ? dv + y * ld : cv + y * kHd;
      unsigned plus = 0, minus = 0;  // bit 4k + e: the value of dimension 8k + 2j + e is +inf or NaN, -inf or NaN
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 v = Type16<T16>::unpack2(reinterpret_cast<const uint32_t*>(v_row)[4 * k + j]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float u = e ? v.y : v.x;
          if (isfinite(u)) continue;
          if (!(u < 0.f)) plus |= 1u << (4 * k + e);
          if (!(u > 0.f)) minus |= 1u << (4 * k + e);
        }
      }
      unsigned open = 0;
#pragma unroll
      for (int g = 0; g < 2; ++g)
        if (i0 + 8 * g + r < x.rows) open |= (plus | minus) << (2 * g);
      if (!__any_sync(0xffffffffu, (open & ~(up & down)) != 0)) continue;
      const uint4 k0 = reinterpret_cast<const uint4*>(k_row + 16 * j)[0],
                  k1 = reinterpret_cast<const uint4*>(k_row + 16 * j)[1];
      const uint32_t kw[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int i = i0 + 8 * g + r;
        const uint4* from = reinterpret_cast<const uint4*>(q_row(a, x, min(i, x.rows - 1)) + 16 * j);
        const uint4 q0 = from[0], q1 = from[1];
        const uint32_t qw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        float s = 0.f;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const float2 qv = Type16<T16>::unpack2(qw[d]), kv = Type16<T16>::unpack2(kw[d]);
          s = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, s));
        }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (i < x.rows) {
          const int t = (x.row0 + i) / a.group;
          const bool seen = p >= len ? (tree.anc[t] >> (p - len)) & 1
                                     : a.window <= 0 || p >= len + tree.depth[t] + 1 - a.window || p < a.sinks;
          const bool none = s == -INFINITY;
          if (seen) {
            up |= (none ? plus | minus : plus) << (2 * g);
            down |= (none ? plus | minus : minus) << (2 * g);
          }
        }
        __syncwarp();
      }
    }
  }
  return (static_cast<unsigned long long>(down) << 32) | up;
}

// Attention of query rows i0 .. i0 + 15 of an item over its tiles j0 .. j0 + cnt - 1 by
// one warp: units at, at + kGroups, ... of them; `first`: of the warps with the same
// units the one that stores drafted K and V; `odd`: there may be values that are not
// finite among them.  False if a wait ran out.
template <typename T16, int WR, bool RIDE>
__device__ __forceinline__ bool attend(const CUtensorMap* map, const DraftArgs<T16>& a, const Item<T16>& x, int i0,
                                       bool first, int at, int j0, int cnt, const Ring<Shape<WR, RIDE>::kUnit>& ring,
                                       Turn<Shape<WR, RIDE>::kSlots>& turn, Tree& tree, Acc& acc, bool& odd) {
  using S = Shape<WR, RIDE>;
  constexpr int U = S::kUnit, kSlots = S::kSlots;
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc.o[i][e] = 0.f;
  acc.m[0] = acc.m[1] = -INFINITY;
  acc.l[0] = acc.l[1] = 0.f;
  const int units = (cnt + U - 1) / U, mine = units > at ? (units - at + S::kGroups - 1) / S::kGroups : 0;
  // a warp with a ring of its own: tiles j0 + at, j0 + at + kGroups, ...
  int row = -1, pos = 0, page = 0, fetched = 0;
  auto next = [&](int slot) {
    if constexpr (!S::kBringer) {
      if ((fetched & 31) == 0) find_tiles(a, x, j0 + at, S::kGroups, fetched, mine, row, pos, page);
      Unit<U> unit;
      unit.row[0] = __shfl_sync(0xffffffffu, row, fetched & 31);
      unit.pos[0] = __shfl_sync(0xffffffffu, pos, fetched & 31);
      const int of[1] = {__shfl_sync(0xffffffffu, page, fetched & 31)};
      ++fetched;
      bring<T16, U>(map, a, x, unit, of, ring, slot);
    }
  };
  if constexpr (!S::kBringer) {
    Turn<kSlots> ahead = turn;
#pragma unroll 1
    for (int s = 0; s < kSlots && fetched < mine; ++s) {
      next(ahead.slot);
      ahead.step(1);
    }
  }
  // q: lane (r, j) holds dimensions 16j..16j+15 of rows r and r + 8
  Query q;
  {
    uint4 f[4] = {};
#pragma unroll
    for (int g = 0; g < (RIDE ? 1 : 2); ++g)
      if (i0 + 8 * g + r < x.rows) {
        const uint4* from = reinterpret_cast<const uint4*>(q_row(a, x, i0 + 8 * g + r) + 16 * j);
        f[2 * g] = from[0];
        f[2 * g + 1] = from[1];
      }
    const uint32_t q_of[4][4] = {{f[0].x, f[2].x, f[0].y, f[2].y},
                                 {f[0].z, f[2].z, f[0].w, f[2].w},
                                 {f[1].x, f[3].x, f[1].y, f[3].y},
                                 {f[1].z, f[3].z, f[1].w, f[3].w}};
#pragma unroll
    for (int i = 0; i < 16; ++i) q.a[i >> 2][i & 3] = q_of[i >> 2][i & 3];
  }
  const bool idle = i0 >= x.rows || mine == 0;  // no rows, or no tiles, for this warp
  // The tree matters where drafted places are, and to a window; it is made while the first tiles are on their
  // way.
  const int last = j0 + cnt - 1;
  const bool drafts = ((last < x.sp.ts ? last : x.sp.tw + last - x.sp.ts) + 1) * kTile > x.sp.len;
  if (lane == 0) tree.odd = 0;
  __syncwarp();
  if ((drafts || a.window > 0) && !idle) build_tree(a, x.b, x.sp, tree);
  Turn<kSlots> now = turn;
  if constexpr (S::kBringer) now.step(at);
  for (int i = 0; i < mine; ++i) {
    const bool ok = mbar_wait(smem_u32(&ring.full[now.slot]), now.parity);
    if (!__all_sync(0xffffffffu, ok)) {
      if (lane == 0) {
        record_error(a.err, kErrTimeout, kSitePagedLoad);
        if constexpr (!S::kBringer)
          for (int s = 0; s < kSlots && i + s < mine; ++s) {  // the loads in flight must not outlive the CTA
            (void)mbar_wait(smem_u32(&ring.full[now.slot]), now.parity);
            now.step(1);
          }
      }
      __syncwarp();
      return false;
    }
    if (!idle) {
      const uint8_t* tiles = ring.buf + now.slot * U * kTileBytes;
      const Unit<U> unit = ring.unit[now.slot];
      if (unit.pos[0] < 0) {
        take<T16, RIDE, false, U>(a, x, i0, q, tiles, unit, tree, acc);
      } else if (unit.row[0] >= 0 || unit.row[U - 1] >= 0) {
        if (first && a.k && x.block == 0) store_drafts(a, x, tiles, unit);
        take<T16, RIDE, true, U>(a, x, i0, q, tiles, unit, tree, acc);
      }
    }
    __syncwarp();
    if constexpr (S::kBringer) {
      if (lane == 0) mbar_arrive(smem_u32(&ring.empty[now.slot]));
      now.step(S::kGroups);
    } else {
      if (lane == 0) fence_proxy_async_smem();
      if (fetched < mine) next(now.slot);
      now.step(1);
    }
  }
  if constexpr (S::kBringer)
    turn.advance(units);
  else
    turn = now;
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
  float any[4] = {0.f, 0.f, 0.f, 0.f};  // NaN if a result is not finite
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) any[e] = fmaf(acc.o[i][e], 0.f, any[e]);
  odd = __any_sync(0xffffffffu, tree.odd != 0 || (any[0] + any[1]) + (any[2] + any[3]) != 0.f);
  return true;
}

// The results that not_finite's bits are of.
__device__ __forceinline__ void put_not_finite(Acc& acc, unsigned long long bits) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool up = (bits >> (4 * i + e)) & 1, down = (bits >> (32 + 4 * i + e)) & 1;
      if (up || down) acc.o[i][e] = up ? (down ? NAN : INFINITY) : -INFINITY;
      if (acc.l[e >> 1] == 0.f) acc.o[i][e] = 0.f;  // nothing but scores of -inf: zeros, whatever the values are
    }
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

__device__ __forceinline__ int rounded(int n, int to) { return to == 1 ? n : (n + to - 1) / to * to; }

// Work is cut into equal runs of tiles over all (sequence, key-value head, row
// block) items laid end to end, one run per CTA, whatever the lengths are.  Where
// there are CTAs enough items are rounded up to whole runs, so that none takes pieces
// of two, one after the other (8 tokens of one sequence of 777, 12 heads: 9.2 us,
// 12.1 without it).  A CTA
// that holds all tiles of an item writes its output, pieces of an item go to the
// workspace and a second kernel joins them.  Groups of warps that took tiles of a
// piece in turn meet in shared memory.
template <typename T16, int WR, bool RIDE>
__global__ void __launch_bounds__((Shape<WR, RIDE>::kThreads), (Shape<WR, RIDE>::kCtas))
    draft_attn(const __grid_constant__ CUtensorMap map, const __grid_constant__ DraftArgs<T16> a) {
  using S = Shape<WR, RIDE>;
  constexpr int kGroups = S::kGroups, kRows = S::kRows, kSlots = S::kSlots, U = S::kUnit;
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_bar[2][S::kRings * kSlots];
  __shared__ __align__(16) Unit<U> s_unit[S::kRings * kSlots];
  __shared__ int s_sum[kWarps], s_whole;
  __shared__ float2 s_ml[kGroups * kRows];
  __shared__ Tree s_tree[kWarps];
  uint8_t* s_tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_meet = s_tiles + (S::kMeetBytes ? S::kRings * S::kRingBytes : 0);
  constexpr int kMeetStep = S::kMeetBytes ? kRows * kHd * 4 : S::kRingBytes;  // from group to group
  int* s_base = reinterpret_cast<int*>(s_tiles + S::kRings * S::kRingBytes + S::kMeetBytes);  // [n_seq + 1]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int of = S::kBringer ? 0 : warp * kSlots;  // this warp's ring
  const Ring<U> ring{s_tiles + of * U * kTileBytes, s_unit + of, s_bar[0] + of, s_bar[1] + of};
  if (tid == 0) {
    for (int s = 0; s < S::kRings * kSlots; ++s) {
      mbar_init(smem_u32(&s_bar[0][s]), 1);
      mbar_init(smem_u32(&s_bar[1][s]), WR);
    }
    fence_barrier_init();
    tma_prefetch_desc(&map);
  }
  griddep_wait();
  // base[b] = tiles of all items of sequences before b, those of an item rounded up to `whole`
  auto count = [&](int whole, bool record) {
    int carry = 0;
    for (int b0 = 0; b0 < a.n_seq; b0 += kTakers) {
      const int b = b0 + tid;
      int v = 0;
      if (tid < kTakers && b < a.n_seq) {
        const Span sp = span_of<kRows>(a, b, record);
        v = rounded(max(sp.nt, 0), whole) * a.n_kv * sp.blocks;
      }
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31 && warp < kWarps) s_sum[warp] = incl;
      __syncthreads();
      int before = carry;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        carry += s_sum[w];
      }
      if (tid < kTakers && b < a.n_seq) s_base[b] = before + incl - v;
      __syncthreads();
    }
    if (tid == 0) s_base[a.n_seq] = carry;
    __syncthreads();
    return carry;
  };
  int total = count(1, blockIdx.x == 0);
  const int grid = static_cast<int>(gridDim.x), run = max((total + grid - 1) / grid, kMinRun);
  const bool few = total <= (grid - min(a.items, grid)) * kMinRun;
  if (tid == 0) s_whole = few ? kMinRun : 1;
  if (few) total = count(kMinRun, false);
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int b = tid; b <= a.n_seq; b += S::kThreads) a.plan[b] = s_base[b];
    if (tid == 0) a.plan[a.n_seq + 1] = few ? -run : run;
  }
  const long long t_first = static_cast<long long>(blockIdx.x) * run;
  if (t_first >= total) return;
  const int t_end = static_cast<int>(min(t_first + run, static_cast<long long>(total)));
  // the piece that begins at t: its item, first tile in it, and tiles
  auto piece_at = [&](int t, int& j0, int& cnt) {
    int lo = 0, hi = a.n_seq;  // last b with base[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_base[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const Span sp = span_of<kRows>(a, lo, false);
    const int nt = rounded(sp.nt, s_whole);
    const int item = (t - s_base[lo]) / nt;
    j0 = (t - s_base[lo]) - item * nt;
    cnt = min(sp.nt - j0, t_end - t);
    return item_of(a, lo, item, sp, kRows);
  };
  Turn<kSlots> turn{0, 0};
  if constexpr (S::kBringer) {
    if (warp == kWarps) {
      bool around = false;
      unsigned by_lanes = 0;
      for (int t = static_cast<int>(t_first); t < t_end;) {
        int j0, cnt;
        const Item<T16> x = piece_at(t, j0, cnt);
        if (!bring_all<T16, U, kSlots>(&map, a, x, j0, cnt, ring, turn, around, by_lanes)) break;
        t = s_whole > 1 ? t_end : t + cnt;
      }
      // copies must not outlive the CTA: each slot's last use, from the oldest on
      for (int s = around ? 0 : kSlots - turn.slot; s < kSlots; ++s) {
        const int slot = (turn.slot + s) % kSlots;
        (void)mbar_wait(smem_u32(&ring.full[slot]), slot < turn.slot ? turn.parity : turn.parity ^ 1);
      }
      return;
    }
  }
  // which units, and which 16 rows: not always the last ones on the same quarter of the SM
  const int at = warp / WR, rank = (warp + static_cast<int>(blockIdx.x)) % WR, i0 = RIDE ? 0 : 16 * rank;
  for (int t = static_cast<int>(t_first); t < t_end;) {
    int j0, cnt;
    const Item<T16> x = piece_at(t, j0, cnt);
    const bool all = cnt == x.sp.nt;
    const long long part = 2ll * blockIdx.x + (t == static_cast<int>(t_first) ? 0 : 1);
    Acc acc;
    bool odd = false;
    const bool ok = attend<T16, WR, RIDE>(&map, a, x, i0, rank == 0, at, j0, cnt, ring, turn, s_tree[warp], acc, odd);
    if (odd) {
      int from, tiles;  // (found again, so that the way to here need not keep them)
      const Item<T16> again = piece_at(t, from, tiles);
      put_not_finite(acc, not_finite<T16, U>(a, again, i0, at, kGroups, from, tiles, s_tree[warp]));
    }
    t = s_whole > 1 ? t_end : t + cnt;
    __syncwarp();
    if constexpr (kGroups == 1) {
      if (!ok) return;
      if (all)
        put_rows(a, x, i0, acc);
      else
        put_piece<T16, RIDE>(acc, x.rows - i0, a.part_o + (part * kRows + i0) * kHd, a.part_ml + part * kRows + i0);
      if (t >= t_end) griddep_launch_dependents();
    } else {
      const int pieces = min((cnt + U - 1) / U, kGroups);
      if (at < pieces && ok)
        put_piece<T16, RIDE>(acc, x.rows - i0, reinterpret_cast<float*>(s_meet + at * kMeetStep) + i0 * kHd,
                             s_ml + at * kRows + i0);
      __syncwarp();
      if (!named_bar_and(ok, 1, kTakers)) return;
      if (t >= t_end) griddep_launch_dependents();
      for (int k = tid; k < x.rows * 16; k += kTakers) {
        const int i = k >> 4, d4 = k & 15;
        float M = -INFINITY, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < pieces; ++w)
          merge<true>(o, M, L, *reinterpret_cast<const float4*>(s_meet + w * kMeetStep + (i * kHd + 4 * d4) * 4),
                s_ml[w * kRows + i]);
        if (all) {
          put_row(a, x, i, d4, o, M, L);
        } else {
          *reinterpret_cast<float4*>(a.part_o + (part * kRows + i) * kHd + 4 * d4) = o;
          if (d4 == 0) a.part_ml[part * kRows + i] = make_float2(M, L);
        }
      }
      // (a ring takes tiles again: generic accesses before asynchronous writes)
      if (!S::kBringer) fence_proxy_async_smem();
      __syncwarp();
      named_bar_sync(1, kTakers);
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
  const int run_few = a.plan[a.n_seq + 1], run = abs(run_few);
  const int start = a.plan[b] + item * (run_few < 0 ? rounded(sp.nt, run) : sp.nt);
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
      for (int u = 0; u < kAhead; ++u) merge<true>(acc, M, L, o[u], ml[u]);
    }
  }
  // pairwise, in an order that the number of threads alone gives
  s_o[tid] = acc;
  s_ml[tid] = make_float2(M, L);
  for (int k = ways >> 1; k > 0; k >>= 1) {
    __syncthreads();
    if (way < k) {
      merge<true>(acc, M, L, s_o[tid + 16 * width * k], s_ml[tid + 16 * width * k]);
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

int ctas_of(int rows) { return rows <= 16 ? Shape<1, false>::kCtas : Shape<2, false>::kCtas; }

template <typename T16, int WR, bool RIDE>
cudaError_t launch_kind(const CUtensorMap& map, DraftArgs<T16> a, cudaStream_t s) {
  using S = Shape<WR, RIDE>;
  constexpr int kFixed = S::kRings * S::kRingBytes + S::kMeetBytes + 1024;
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
  const int sms = num_sms(), max_blocks = (a.T * a.group + S::kRows - 1) / S::kRows;
  const long long items = static_cast<long long>(a.n_seq) * a.n_kv * max_blocks;
  a.items = static_cast<int>(std::min(items, 1ll << 30));
  cudaError_t e = launch_pdl(draft_attn<T16, WR, RIDE>, sms * S::kCtas, S::kThreads, kFixed + (a.n_seq + 1) * 4, s, 0,
                             map, a);
  if (e != cudaSuccess) return e;
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
  const size_t slots = 2ull * num_sms() * ctas_of(rows) * rows;
  char* base = static_cast<char*>(ws);
  a.plan = reinterpret_cast<int*>(base);
  base += align256((static_cast<size_t>(c->n_seq) + 2) * 4);
  a.part_ml = reinterpret_cast<float2*>(base);
  base += align256(slots * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(base);
  a.n_layer = c->n_layer;
  a.layer = layer;
  // the pool: dimensions, rows of all heads, K or V, layers of pages; a box is a tile's K and V
  const uint64_t rows_kv = static_cast<uint64_t>(c->n_kv_head) * c->page_size, row_bytes = kHd * 2;
  CUtensorMap map;
  if (!encode_tma_4d(&map, Type16<T16>::kTma, c->pages,
                     {kHd, rows_kv, 2, static_cast<uint64_t>(c->n_pages) * c->n_layer},
                     {row_bytes, rows_kv * row_bytes, 2 * rows_kv * row_bytes}, {kHd, kTile, 2, 1}))
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
  const int rows = rows_of(T, n_head / c->n_kv_head);
  const size_t slots = 2ull * num_sms() * ctas_of(rows) * rows;
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
