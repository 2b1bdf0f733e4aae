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
// the tensor cores need to be the limit, and what a row costs beside its
// products (two roundings of p, its exponential, maximum and sum: about nine
// instructions a score and lane) is what the rows pay for on either kind of
// matrix instruction.  So the products are mma.sync m16n8k16 with rows in blocks
// of 16, whose results stay in registers, and the layout serves the loads: each
// warp runs its own ring of TMA boxes (16 rows of K, 16 of V).
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
constexpr int kStageBytes = 2 * kBoxBytes;  // K, then V
constexpr int kMinRun = 2 * kWarps;         // tiles per CTA at least

// NB: blocks of 16 query rows.  RIDE: up to 8 rows in one block, whose other 8
// carry the rounding remainder of p.
template <int NB, bool RIDE>
struct Shape {
  static constexpr int kRows = RIDE ? 8 : 16 * NB;
  // a warp's result (fp32 rows of 64) takes the place of its ring
  static constexpr int kStages = NB >= 4 ? 4 : 2;
  static constexpr int kCtasPerSm = NB >= 4 ? 2 : NB == 2 ? 3 : 4;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr bool kSharedQ = NB >= 4;  // the query rows in shared memory, not in registers
  static_assert(kRingBytes >= kRows * kHd * 4, "a warp's result fits its ring");
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

// A warp's ring of tiles.
struct Ring {
  const CUtensorMap* map;
  uint8_t* buf;   // [stages][K box, V box], 1024-byte aligned
  uint64_t* bar;  // [stages]
  int slot, parity;  // of the tile to take next
};

// What one warp makes of its tiles of one item: o (not divided by l), m (log2
// units) and l of its query rows.  Lane (r = lane / 4, j = lane % 4) holds rows
// r and r + 8 of each block: o[i] their dimensions 16j + i and 16j + 8 + i.
template <int NB>
struct Acc {
  float o[NB][8][4];
  float m[NB][2], l[NB][2];
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
__device__ __forceinline__ bool finite2(uint32_t w) {
  constexpr uint32_t kExp = std::is_same<T16, __half>::value ? 0x7c00u : 0x7f80u;
  return (w & kExp) != kExp && ((w >> 16) & kExp) != kExp;
}
template <typename T16>
__device__ __forceinline__ uint32_t only_finite2(uint32_t w) {
  constexpr uint32_t kExp = std::is_same<T16, __half>::value ? 0x7c00u : 0x7f80u;
  if ((w & kExp) == kExp) w &= 0xffff0000u;
  if (((w >> 16) & kExp) == kExp) w &= 0xffffu;
  return w;
}

// fp16 p times a value that is not finite (of place `at` of the tile whose
// values are vb): what the products with zero in that place have left out.
template <typename T16, int NB, bool RIDE>
__device__ __forceinline__ void add_not_finite(Acc<NB>& acc, int blk, const float (&s)[2][4], const uint8_t* vb,
                                               int places) {
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
    for (int e = 0; e < 2; ++e) {
      const uint4 u = *reinterpret_cast<const uint4*>(vb + at * 128 + (((2 * j + e) ^ (at & 7)) << 4));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (finite2<T16>(w[i])) continue;
        const float2 v = Type16<T16>::unpack2(w[i]);
#pragma unroll
        for (int g = 0; g < (RIDE ? 1 : 2); ++g) {
          if (p[g] < 0.f) continue;  // not visible
          if (!isfinite(v.x)) acc.o[blk][2 * i][2 * g + e] += p[g] * v.x;
          if (!isfinite(v.y)) acc.o[blk][2 * i + 1][2 * g + e] += p[g] * v.y;
        }
      }
    }
  }
}

// Attention of an item's query rows over its tiles j0, j0 + step, ... (cnt of
// them) by one warp.  False if a wait ran out.  s_q: the query rows in shared
// memory (Shape::kSharedQ), swizzled as a tile is.
//
// The B fragments of both products come out of shared memory as they are: sums
// over dimensions and the order of output dimensions are free, so lane (r, j)
// reads of key rows r and r + 8 the dimensions 16j..16j+15 (q alike) and of value
// rows 2j, 2j+1, 2j+8, 2j+9 the dimensions 8r..8r+7, where output column r of
// product i stands for dimension 8r + i.  With the boxes' 128-byte swizzle
// (16-byte unit u of row x at u ^ (x & 7)) no bank is read twice in a phase.
//
// Tiles with places behind the cached positions are brought by the lanes
// (16-byte asynchronous copies): cached places from their page, drafted ones
// from k and v, which are also stored in the page from here.
template <typename T16, int NB, bool RIDE>
__device__ __forceinline__ bool attend(const DraftArgs<T16>& a, const Item<T16>& x, int j0, int step, int cnt,
                                       Ring& ring, const uint8_t* s_q, Tree& tree, Acc<NB>& acc) {
  using S = Shape<NB, RIDE>;
  constexpr int kStages = S::kStages;
  constexpr int kHalves = RIDE ? 1 : 2;  // row groups of a lane that hold rows
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int len = x.sp.len, end = len + x.sp.n;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc.o[b][i][e] = 0.f;
    acc.m[b][0] = acc.m[b][1] = -INFINITY;
    acc.l[b][0] = acc.l[b][1] = 0.f;
  }
  auto tile_no = [&](int i) {
    const int t = j0 + i * step;
    return t < x.sp.ts ? t : x.sp.tw + (t - x.sp.ts);
  };
  // lane i: first row (K) of tile (i + a multiple of 32) of this run, -1 when its page is not there
  int rows32 = -1, fetched = 0;
  auto issue = [&](int i, int slot) {
    if ((i & 31) == 0) {
      rows32 = -1;
      if (i + lane < cnt) {
        const int pos = tile_no(i + lane) * kTile, c = pos / a.page_size;
        const int page = x.pages[c];
        if (page >= 0 && page < a.n_pages)
          rows32 = page * a.page_rows + a.row0 + x.kvh * a.page_size + (pos - c * a.page_size);
        else
          record_error(a.err, kErrRange, kSitePagedPage);
      }
    }
    const int row = __shfl_sync(0xffffffffu, rows32, i & 31);
    const uint32_t bar = smem_u32(&ring.bar[slot]), dst = smem_u32(ring.buf + slot * kStageBytes);
    const int pos0 = tile_no(i) * kTile;
    if (row >= 0 && a.k && pos0 + kTile > len) {  // (the same for all lanes)
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = (lane >> 3) + 4 * (u & 3), c = lane & 7, part = u >> 2, p = pos0 + at;
        const T16* from = nullptr;
        if (p < len)
          from = a.pages + (static_cast<long long>(row - a.row0) + at + part * a.n_kv * a.page_size) * kHd + c * 8;
        else if (p < end)
          from = (part ? a.v : a.k) + (static_cast<long long>(x.b) * a.T + (p - len)) * a.ldkv + x.kvh * kHd + c * 8;
        if (from)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + part * kBoxBytes + at * 128 +
                                                                         ((c ^ (at & 7)) << 4)),
                       "l"(from)
                       : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    } else if (lane == 0) {
      if (row >= 0) {
        mbar_arrive_expect_tx(bar, kStageBytes);
        tma_load_2d(dst, ring.map, bar, 0, row);
        tma_load_2d(dst + kBoxBytes, ring.map, bar, 0, row + a.n_kv * a.page_size);
      } else {
        mbar_arrive(bar);  // nothing to wait for
      }
    }
    return row;
  };
  int rows[kStages];  // of the tiles in the ring, oldest first
  int slot = ring.slot;
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    rows[s] = -1;
    if (fetched < cnt) {
      rows[s] = issue(fetched, slot);
      ++fetched;
      slot = slot + 1 == kStages ? 0 : slot + 1;
    }
  }
  // q: lane (r, j) holds dimensions 16j..16j+15 of rows r and r + 8 of each block
  uint4 qf[S::kSharedQ ? 1 : NB][4] = {};
  if constexpr (!S::kSharedQ) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int g = 0; g < kHalves; ++g)
        if (16 * b + 8 * g + r < x.rows) {
          const uint4* from = reinterpret_cast<const uint4*>(q_row(a, x, 16 * b + 8 * g + r) + 16 * j);
          qf[b][2 * g] = from[0];
          qf[b][2 * g + 1] = from[1];
        }
  }
  bool have_tree = false;

  for (int i = 0; i < cnt; ++i) {
    const bool ok = mbar_wait(smem_u32(&ring.bar[ring.slot]), ring.parity);
    if (!__all_sync(0xffffffffu, ok)) {
      if (lane == 0) {
        record_error(a.err, kErrTimeout, kSitePagedLoad);
        for (int s = 0; s < kStages && i + s < cnt; ++s) {  // the loads in flight must not outlive the CTA
          const int k = ring.slot + s;
          (void)mbar_wait(smem_u32(&ring.bar[k % kStages]), ring.parity ^ (k >= kStages ? 1 : 0));
        }
      }
      __syncwarp();
      return false;
    }
    uint8_t* kb = ring.buf + ring.slot * kStageBytes;
    uint8_t* vb = kb + kBoxBytes;
    const int row = rows[0], pos0 = tile_no(i) * kTile;
    if (row >= 0) {
      // a tile that every row sees all of
      const bool whole = pos0 + kTile <= len && (a.window <= 0 || pos0 >= end - a.window || pos0 + kTile <= a.sinks);
      if (!whole && !have_tree) {
        build_tree(a, x.b, x.sp, tree);
        have_tree = true;
      }
      if (a.k && x.block == 0 && pos0 + kTile > len) {  // the drafted tokens' K and V into their page
        const int page = x.pages[pos0 / a.page_size];
        if (a.refs[page] > 1) {  // not into a page that other sequences read
          if (lane == 0) record_error(a.err, kErrRange, kSitePagedShared);
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int at = (lane >> 3) + 4 * (u & 3), c = lane & 7, part = u >> 2, p = pos0 + at;
            if (p >= len && p < end)
              *reinterpret_cast<uint4*>(
                  a.pages + (static_cast<long long>(row - a.row0) + at + part * a.n_kv * a.page_size) * kHd + c * 8) =
                  *reinterpret_cast<const uint4*>(kb + part * kBoxBytes + at * 128 + ((c ^ (at & 7)) << 4));
          }
        }
      }
      uint4 kf[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint8_t* kr = kb + (r + 8 * e) * 128;
        kf[e][0] = *reinterpret_cast<const uint4*>(kr + (((2 * j) ^ r) << 4));
        kf[e][1] = *reinterpret_cast<const uint4*>(kr + (((2 * j + 1) ^ r) << 4));
      }
      uint32_t vf[8][2];
      bool odd = false;  // a value that is not finite, in a tile that not every row sees all of
      {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int vr = 2 * j + (e & 1) + (e >> 1) * 8;
          v[e] = *reinterpret_cast<const uint4*>(vb + vr * 128 + ((r ^ (vr & 7)) << 4));
          if (!whole) {
            if (pos0 + vr >= end) v[e] = make_uint4(0, 0, 0, 0);  // nothing wrote it: it may hold anything
            odd |= !(finite2<T16>(v[e].x) && finite2<T16>(v[e].y) && finite2<T16>(v[e].z) && finite2<T16>(v[e].w));
          }
        }
        if (!whole) {
          odd = __any_sync(0xffffffffu, odd);
          if (odd)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = make_uint4(only_finite2<T16>(v[e].x), only_finite2<T16>(v[e].y), only_finite2<T16>(v[e].z),
                                only_finite2<T16>(v[e].w));
        }
        const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&v[0]);
        const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&v[1]);
        const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&v[2]);
        const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&v[3]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t sel = (k & 1) ? 0x7632u : 0x5410u;
          vf[k][0] = __byte_perm(v0[k >> 1], v1[k >> 1], sel);
          vf[k][1] = __byte_perm(v2[k >> 1], v3[k >> 1], sel);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (NB > 1 && 16 * b >= x.rows) break;
        uint4 q0, q1, q2, q3;  // rows r (its two halves), r + 8
        if constexpr (S::kSharedQ) {
          const uint8_t* qr = s_q + (16 * b + r) * 128;
          q0 = *reinterpret_cast<const uint4*>(qr + (((2 * j) ^ r) << 4));
          q1 = *reinterpret_cast<const uint4*>(qr + (((2 * j + 1) ^ r) << 4));
          q2 = *reinterpret_cast<const uint4*>(qr + 1024 + (((2 * j) ^ r) << 4));
          q3 = *reinterpret_cast<const uint4*>(qr + 1024 + (((2 * j + 1) ^ r) << 4));
        } else {
          q0 = qf[b][0], q1 = qf[b][1], q2 = qf[b][2], q3 = qf[b][3];
        }
        float s[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[e][0] = s[e][1] = s[e][2] = s[e][3] = 0.f;
          mma16816<T16>(s[e], q0.x, q2.x, q0.y, q2.y, kf[e][0].x, kf[e][0].y);
          mma16816<T16>(s[e], q0.z, q2.z, q0.w, q2.w, kf[e][0].z, kf[e][0].w);
          mma16816<T16>(s[e], q1.x, q3.x, q1.y, q3.y, kf[e][1].x, kf[e][1].y);
          mma16816<T16>(s[e], q1.z, q3.z, q1.w, q3.w, kf[e][1].z, kf[e][1].w);
        }
        uint32_t hidden = 0;  // bit 4e + 2g + k: score s[e][2g + k] is not visible
        if (!whole) {
#pragma unroll
          for (int g = 0; g < kHalves; ++g) {
            const int i_row = min(16 * b + 8 * g + r, x.rows - 1);
            const int t = (x.row0 + i_row) / a.group;
            const unsigned long long anc = tree.anc[t];
            const int first = a.window > 0 ? len + tree.depth[t] + 1 - a.window : 0;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int p = pos0 + 8 * e + 2 * j + k;
                const bool seen = p < len ? (p >= first || p < a.sinks) : p < end && ((anc >> (p - len)) & 1);
                if (!seen) {
                  s[e][2 * g + k] = -INFINITY;
                  hidden |= 1u << (4 * e + 2 * g + k);
                }
              }
          }
        }
        float alpha[2] = {1.f, 1.f};
#pragma unroll
        for (int g = 0; g < kHalves; ++g) {
          float mx = fmaxf(fmaxf(s[0][2 * g], s[0][2 * g + 1]), fmaxf(s[1][2 * g], s[1][2 * g + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(acc.m[b][g], mx * a.scale_log2);
          const float ms = mn == -INFINITY ? 0.f : mn;  // every score so far is -inf
          alpha[g] = acc.m[b][g] == mn ? 1.f : ex2_approx(acc.m[b][g] - ms);
          acc.m[b][g] = mn;
          const float bias = kShift<T16> - ms;
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < 2; ++k) s[e][2 * g + k] = ex2_approx(fmaf(s[e][2 * g + k], a.scale_log2, bias));
          acc.l[b][g] = fmaf(acc.l[b][g], alpha[g], (s[0][2 * g] + s[0][2 * g + 1]) + (s[1][2 * g] + s[1][2 * g + 1]));
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            acc.o[b][k][0] *= alpha[0];
            acc.o[b][k][1] *= alpha[0];
            acc.o[b][k][2] *= alpha[RIDE ? 0 : 1];
            acc.o[b][k][3] *= alpha[RIDE ? 0 : 1];
          }
        }
        uint32_t ph[2][2], pl[2][2];  // [position half][row half]
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int g = 0; g < kHalves; ++g) split2<T16>(s[e][2 * g], s[e][2 * g + 1], ph[e][g], pl[e][g]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if constexpr (RIDE) {
            mma16816<T16>(acc.o[b][k], ph[0][0], pl[0][0], ph[1][0], pl[1][0], vf[k][0], vf[k][1]);
          } else {
            mma16816<T16>(acc.o[b][k], ph[0][0], ph[0][1], ph[1][0], ph[1][1], vf[k][0], vf[k][1]);
            mma16816<T16>(acc.o[b][k], pl[0][0], pl[0][1], pl[1][0], pl[1][1], vf[k][0], vf[k][1]);
          }
        }
        if (odd) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if ((hidden >> (4 * e + k)) & 1) s[e][k] = -1.f;
          add_not_finite<T16, NB, RIDE>(acc, b, s, vb, min(kTile, end - pos0));
        }
      }
    }
    // the slot is read: the tile kStages further on
    __syncwarp();
    if (lane == 0) fence_proxy_async_smem();
#pragma unroll
    for (int s = 0; s + 1 < kStages; ++s) rows[s] = rows[s + 1];
    rows[kStages - 1] = -1;
    if (fetched < cnt) {
      rows[kStages - 1] = issue(fetched, ring.slot);
      ++fetched;
    }
    if (++ring.slot == kStages) {
      ring.slot = 0;
      ring.parity ^= 1;
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {  // sums over the four lanes of a row
      acc.l[b][g] += __shfl_xor_sync(0xffffffffu, acc.l[b][g], 1);
      acc.l[b][g] += __shfl_xor_sync(0xffffffffu, acc.l[b][g], 2);
    }
    if (RIDE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc.o[b][i][0] += acc.o[b][i][2];
        acc.o[b][i][1] += acc.o[b][i][3];
      }
    }
  }
  return true;
}

// The rows of one warp's result: dst[row][64], ml[row] = (m, l).
template <typename T16, int NB, bool RIDE>
__device__ __forceinline__ void put_piece(const Acc<NB>& acc, int rows, float* dst, float2* ml) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int g = 0; g < (RIDE ? 1 : 2); ++g) {
      const int i = 16 * b + 8 * g + r;
      if (i >= rows) continue;
      float* po = dst + i * kHd + 16 * j;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        *reinterpret_cast<float4*>(po + 8 * e) = make_float4(acc.o[b][0][2 * g + e], acc.o[b][1][2 * g + e],
                                                             acc.o[b][2][2 * g + e], acc.o[b][3][2 * g + e]);
        *reinterpret_cast<float4*>(po + 8 * e + 4) = make_float4(acc.o[b][4][2 * g + e], acc.o[b][5][2 * g + e],
                                                                 acc.o[b][6][2 * g + e], acc.o[b][7][2 * g + e]);
      }
      if (j == 0) ml[i] = make_float2(acc.m[b][g] - kShift<T16>, acc.l[b][g]);
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
// block) items laid end to end, one run per CTA, whatever the lengths are.  The
// warps of a CTA take the tiles of an item in turn and meet in shared memory; a
// CTA that holds all tiles of an item writes its output, pieces of an item go to
// the workspace and a second kernel joins them.
template <typename T16, int NB, bool RIDE>
__global__ void __launch_bounds__(kThreads, (Shape<NB, RIDE>::kCtasPerSm))
    draft_attn(const __grid_constant__ CUtensorMap map, const DraftArgs<T16> a) {
  using S = Shape<NB, RIDE>;
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_bar[kWarps * S::kStages];
  __shared__ int s_sum[kWarps];
  __shared__ float2 s_ml[kWarps * S::kRows];
  __shared__ Tree s_tree[kWarps];
  uint8_t* s_tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = s_tiles + kWarps * S::kRingBytes;
  int* s_base = reinterpret_cast<int*>(s_q + (S::kSharedQ ? S::kRows * 128 : 0));  // [n_seq + 1]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Ring ring{&map, s_tiles + warp * S::kRingBytes, s_bar + warp * S::kStages, 0, 0};
  if (lane == 0) {
    for (int s = 0; s < S::kStages; ++s) mbar_init(smem_u32(&ring.bar[s]), 1);
    fence_barrier_init();
    tma_prefetch_desc(&map);
  }
  __syncwarp();
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
    if constexpr (S::kSharedQ) {
      for (int i = tid; i < S::kRows * 8; i += kThreads) {
        const int row = i >> 3, c = i & 7;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (row < x.rows) u = *reinterpret_cast<const uint4*>(q_row(a, x, row) + 8 * c);
        *reinterpret_cast<uint4*>(s_q + row * 128 + ((c ^ (row & 7)) << 4)) = u;
      }
      __syncthreads();
    }
    bool ok = true;
    {
      Acc<NB> acc;
      const int mine = cnt > warp ? (cnt - warp + kWarps - 1) / kWarps : 0;
      if (mine > 0) {
        ok = attend<T16, NB, RIDE>(a, x, j0 + warp, kWarps, mine, ring, s_q, s_tree[warp], acc);
        __syncwarp();
        if (ok)
          put_piece<T16, NB, RIDE>(acc, x.rows, reinterpret_cast<float*>(ring.buf), s_ml + warp * S::kRows);
      }
    }
    if (!__syncthreads_and(ok)) return;
    t += cnt;
    if (t >= t_end) griddep_launch_dependents();
    const bool all = cnt == sp.nt;
    const int pieces = min(cnt, kWarps);
    const long long part = 2ll * blockIdx.x + (t - cnt == static_cast<int>(t_first) ? 0 : 1);
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
    if (t < t_end) {
      // the rings take tiles again: generic reads before asynchronous writes
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

// Query rows per block, and what follows from them, for T tokens of a group of
// heads: few rows leave registers for more warps (and, up to 8, carry the
// remainder of p for nothing), more of them read the cache less often.
struct Plan {
  int kind;  // 0: 8 rows, 1: 16, 2: 32, 3: 64
  int rows, ctas_per_sm;
};
Plan plan_of(int T, int group) {
  const int rows = T * group;
  if (rows <= 8) return {0, 8, Shape<1, true>::kCtasPerSm};
  if (rows <= 16) return {1, 16, Shape<1, false>::kCtasPerSm};
  if (rows <= 32) return {2, 32, Shape<2, false>::kCtasPerSm};
  return {3, 64, Shape<4, false>::kCtasPerSm};
}

template <typename T16, int NB, bool RIDE>
cudaError_t launch_kind(const CUtensorMap& map, const DraftArgs<T16>& a, cudaStream_t s) {
  using S = Shape<NB, RIDE>;
  const int fixed = kWarps * S::kRingBytes + 1024 + (S::kSharedQ ? S::kRows * 128 : 0);
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(draft_attn<T16, NB, RIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         fixed + (kMaxPagedSeqs + 1) * 4);
    if (e != cudaSuccess) return e;
    // the join leaves the SMs split as draft_attn has them: between two splits an SM has to run empty
    e = cudaFuncSetAttribute(draft_join<T16, S::kRows>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  const int sms = num_sms();
  cudaError_t e = launch_pdl(draft_attn<T16, NB, RIDE>, sms * S::kCtasPerSm, kThreads, fixed + (a.n_seq + 1) * 4, s, 0,
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
  const Plan p = plan_of(T, a.group);
  const size_t slots = 2ull * num_sms() * p.ctas_per_sm * p.rows;
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
  switch (p.kind) {
    case 0: return launch_kind<T16, 1, true>(map, a, s);
    case 1: return launch_kind<T16, 1, false>(map, a, s);
    case 2: return launch_kind<T16, 2, false>(map, a, s);
    default: return launch_kind<T16, 4, false>(map, a, s);
  }
}

}  // namespace

size_t attention_draft_workspace(const gpt2_paged_cache* c, int T, int n_head) {
  const Plan p = plan_of(T, n_head / c->n_kv_head);
  const size_t slots = 2ull * num_sms() * p.ctas_per_sm * p.rows;
  return align256((static_cast<size_t>(c->n_seq) + 2) * 4) + align256(slots * sizeof(float2)) +
         align256(slots * kHd * 4);
}

bool attention_draft_fits(const gpt2_paged_cache* c, int T, int n_head) {
  // rows of the pool are TMA coordinates, and tiles of all items are counted, in
  // 32 bits, the latter with room for one run more
  if (static_cast<double>(c->n_pages) * c->n_layer * 2 * c->n_kv_head * c->page_size >= 2147483648.0) return false;
  const Plan p = plan_of(T, n_head / c->n_kv_head);
  const long long blocks = (static_cast<long long>(T) * (n_head / c->n_kv_head) + p.rows - 1) / p.rows;
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
