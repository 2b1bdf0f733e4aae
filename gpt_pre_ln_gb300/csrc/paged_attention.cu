// Attention of one new token per sequence over a paged key-value cache
// (16-bit paths), optionally under a sliding window with a few first
// positions that stay visible.
//
//   out[b, h] = sum_{p visible} softmax_p(c q_h . k_p) v_p
//
// with n positions (the cached ones and, when it is given, the new token at
// position n - 1) of which p is visible when p >= n - window or p < sinks (all
// of them without a window).  Query head h reads key-value head
// h / (n_head / n_kv_head).
//
// With up to 16 query heads to a key-value head every visible key and value row
// is read once (256 bytes a position and key-value head) and takes 4 * 64 flop
// per query head: at most 16 flop a byte, far under what the tensor cores need
// to be the limit, so the kernel is bound by HBM bandwidth and its layout serves
// the loads: each warp runs its own ring of TMA boxes (16 rows of K, 16 of V),
// 128 KB of them on an SM, and waits for nobody else.  The products
// are mma.sync m16n8k16 with the few query heads as rows: a tcgen05 tile would
// be 128 rows, its operands shared by four warps, and the kernel has no use for
// the rate.
//
// More query heads are cut into even blocks of at most 16, each of which reads all
// of its key-value head again, from L2 or, in a long cache, from HBM: 64 sequences
// of 32000 positions in bf16 (524 MB) take 115 us with 16 heads on 1, 170 with 25
// and 289 with 40 (two and three blocks); of 4000 (66 MB, within L2) 29, 35 and 57.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace gpt2 {

namespace {

constexpr int kHd = 64;
constexpr int kTile = 16;    // positions per tile; page sizes are multiples of it
constexpr int kWarps = 4;    // warps per CTA, independent of one another
constexpr int kCtasPerSm = 4;
constexpr int kStages = 2;   // tiles per warp in flight or in use
constexpr int kMinRun = 2;   // tiles per warp at least; twice that where a piece of 9 or more heads weighs as much
constexpr int kBoxBytes = kTile * kHd * 2;
constexpr int kStageBytes = 2 * kBoxBytes;  // K, then V
constexpr int kWarpBytes = kStages * kStageBytes;
static_assert(kWarpBytes >= 16 * kHd * 4, "a warp's result fits its ring");

template <typename T16>
struct PagedArgs {
  const T16* q;
  const T16* k_new;  // null: the query attends over the cached positions only
  const T16* v_new;
  T16* out;
  float* lse;  // nullable, [n_seq, H]
  T16* pages;  // the layer's part of page 0
  int row0, page_rows;  // the pool as rows of 64: the layer's first row, rows per page
  const int32_t* table;
  const int32_t* lens;
  const int32_t* refs;
  int* plan;       // base[n_seq + 1], then tiles per warp
  float* part_o;   // [2 * warps, HB, 64]
  float2* part_ml;  // [2 * warps, HB]: running maximum (log2 units) and sum
  unsigned* err;
  long long ldq, ldkv, ldo;
  int n_pages, page_size, max_pages, n_seq, n_kv, H, group;
  int n_hb, HB;  // blocks of query heads per key-value head, heads per block
  int window, sinks;
  float scale_log2;  // score scale times log2(e)
};

// The tiles that one sequence's query sees: [0, ts) and [tw, tw + nt - ts).
// nt < 0: the slot is idle (or its length does not fit its table) and its row
// of the output is left alone.
struct Span {
  int n, ts, tw, nt;
};
template <typename T16>
__device__ __forceinline__ Span span_of(const PagedArgs<T16>& a, int b, bool record) {
  const int len = a.lens[b], more = a.k_new ? 1 : 0;
  Span s{0, 0, 0, -1};
  if (len < 0) return s;
  if (len > a.max_pages * a.page_size - more) {
    if (record) record_error(a.err, kErrRange, kSitePagedLength);
    return s;
  }
  const int n = len + more;
  s.n = n;
  const int te = (n + kTile - 1) / kTile;
  if (a.window > 0 && n > a.window) {
    const int first = n - a.window;
    s.tw = first / kTile;
    s.ts = min((min(a.sinks, first) + kTile - 1) / kTile, s.tw);
  }
  s.nt = s.ts + te - s.tw;
  return s;
}

template <typename T16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T16, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (p rounded, what that lost) in 16 bits, so that their sum carries p to 16
// bits (bf16) or 22 bits (fp16).  In bf16 that moves 2 of 1000 output elements, those
// next to a border, to the neighbouring bf16 number (fp32 sums in another order
// move 0.3); the error against 64 bits stays that of the result's own rounding,
// 1.7e-3.  A third bf16 part left 0.3 to 1.1 and cost 2.4% under a window at 25 heads.
template <typename T16>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = Type16<T16>::pack2(x, y);
  const float2 h = Type16<T16>::unpack2(hi);
  lo = Type16<T16>::pack2(x - h.x, y - h.y);
}

// A warp's ring of tiles.
struct Ring {
  const CUtensorMap* map;
  uint8_t* buf;   // [kStages][K box, V box], 1024-byte aligned
  uint64_t* bar;  // [kStages]
  int slot, parity;  // of the tile to take next
};

// What one warp makes of a run of tiles of one item: o (not divided by l), m
// (log2 units) and l of its query heads.  Lane (r = lane / 4, j = lane % 4)
// holds head r (and r + 8 when WIDE, in the upper halves): o[i] its dimensions
// 16j + i and 16j + 8 + i.
struct Acc {
  float o[8][4];
  float m[2], l[2];
};

// Where an item's keys, values and queries are.
template <typename T16>
struct Item {
  Span sp;
  const int32_t* pages;  // the sequence's table row
  const T16* q;          // its first query head
  const T16* k_new;      // the new token's rows of this key-value head
  const T16* v_new;
  int b, kvh, hb, head0, heads;
};

template <typename T16>
__device__ __forceinline__ Item<T16> item_of(const PagedArgs<T16>& a, int b, int item, const Span& sp) {
  Item<T16> x;
  x.sp = sp;
  x.b = b;
  x.kvh = item / a.n_hb;
  x.hb = item - x.kvh * a.n_hb;
  x.head0 = x.kvh * a.group + x.hb * a.HB;
  x.heads = min(a.HB, a.group - x.hb * a.HB);
  x.pages = a.table + static_cast<long long>(b) * a.max_pages;
  x.q = a.q + b * a.ldq + static_cast<long long>(x.head0) * kHd;
  x.k_new = a.k_new ? a.k_new + b * a.ldkv + x.kvh * kHd : nullptr;
  x.v_new = a.k_new ? a.v_new + b * a.ldkv + x.kvh * kHd : nullptr;
  return x;
}

// fp16 probabilities are carried 2^12 times larger: their smallest step is then
// 2^-36 of the row's largest and not 2^-24.
template <typename T16>
constexpr float kShift = std::is_same<T16, __half>::value ? 12.f : 0.f;

// Attention of an item's query heads over its tiles j0, j0 + step, ... (cnt of
// them) by one warp.  False if a wait ran out.
//
// The B fragments of both products come out of shared memory as they are:
// sums over dimensions and the order of output dimensions are free, so lane
// (r, j) reads of key rows r and r + 8 the dimensions 16j..16j+15 (q is loaded
// alike) and of value rows 2j, 2j+1, 2j+8, 2j+9 the dimensions 8r..8r+7, where
// output column r of product i stands for dimension 8r + i.  With the boxes'
// 128-byte swizzle (16-byte unit u of row x at u ^ (x & 7)) the eight lanes of
// a 16-byte access phase touch eight different units, so no bank twice.
//
// WIDE: 9 to 16 query heads fill the 16 rows of the A operand; the rounding
// remainder of p then takes a second product.  Up to 8 heads leave rows 8..15
// free and the remainder rides there.
template <typename T16, bool WIDE>
__device__ __forceinline__ bool attend(const PagedArgs<T16>& a, const Item<T16>& x, int j0, int step, int cnt,
                                       Ring& ring, Acc& acc) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int n = x.sp.n, pos_new = x.k_new ? n - 1 : -1;
  constexpr int kRows = WIDE ? 2 : 1;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc.o[i][e] = 0.f;
  acc.m[0] = acc.m[1] = -INFINITY;
  acc.l[0] = acc.l[1] = 0.f;
  auto tile_no = [&](int i) {
    const int t = j0 + i * step;
    return t < x.sp.ts ? t : x.sp.tw + (t - x.sp.ts);
  };
  // lane i: first row (K) of tile (i + a multiple of 32) of this run, -1 when
  // its page is not there
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
    if (lane == 0) {
      const uint32_t bar = smem_u32(&ring.bar[slot]), dst = smem_u32(ring.buf + slot * kStageBytes);
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
  // q: lane (r, j) holds dimensions 16j..16j+15 of rows r (and r + 8)
  uint4 qa[2] = {}, qb[2] = {};
  if (r < x.heads) {
    qa[0] = *reinterpret_cast<const uint4*>(x.q + static_cast<long long>(r) * kHd + 16 * j);
    qa[1] = *reinterpret_cast<const uint4*>(x.q + static_cast<long long>(r) * kHd + 16 * j + 8);
  }
  if (WIDE && r + 8 < x.heads) {
    qb[0] = *reinterpret_cast<const uint4*>(x.q + static_cast<long long>(r + 8) * kHd + 16 * j);
    qb[1] = *reinterpret_cast<const uint4*>(x.q + static_cast<long long>(r + 8) * kHd + 16 * j + 8);
  }
  // the new token's row: lanes 0..7 its key, 8..15 its value, 16 bytes each
  uint4 fresh = make_uint4(0, 0, 0, 0);
  const bool has_new = pos_new >= 0 && j0 + (cnt - 1) * step == x.sp.nt - 1;
  if (has_new && lane < 16) fresh = *(reinterpret_cast<const uint4*>(lane < 8 ? x.k_new : x.v_new) + (lane & 7));
  bool store = has_new && x.hb == 0;
  if (store) {  // not into a page that other sequences read
    const int page = x.pages[pos_new / a.page_size];
    if (page >= 0 && page < a.n_pages && a.refs[page] > 1) {
      if (lane == 0) record_error(a.err, kErrRange, kSitePagedShared);
      store = false;
    }
  }
  auto visible = [&](int p) { return p < n && (a.window <= 0 || p >= n - a.window || p < a.sinks); };

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
    if (has_new && i == cnt - 1 && row >= 0) {
      const int at = pos_new - pos0;
      if (lane < 16) {
        *reinterpret_cast<uint4*>((lane < 8 ? kb : vb) + at * 128 + (((lane & 7) ^ (at & 7)) << 4)) = fresh;
        if (store) {
          T16* to = a.pages + (static_cast<long long>(row - a.row0) + at + (lane < 8 ? 0 : a.n_kv * a.page_size)) * kHd;
          *reinterpret_cast<uint4*>(to + (lane & 7) * 8) = fresh;
        }
      }
      __syncwarp();
    }
    if (row >= 0) {
      float s[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint8_t* kr = kb + (r + 8 * e) * 128;
        const uint4 k0 = *reinterpret_cast<const uint4*>(kr + (((2 * j) ^ r) << 4));
        const uint4 k1 = *reinterpret_cast<const uint4*>(kr + (((2 * j + 1) ^ r) << 4));
        s[e][0] = s[e][1] = s[e][2] = s[e][3] = 0.f;
        mma16816<T16>(s[e], qa[0].x, qb[0].x, qa[0].y, qb[0].y, k0.x, k0.y);
        mma16816<T16>(s[e], qa[0].z, qb[0].z, qa[0].w, qb[0].w, k0.z, k0.w);
        mma16816<T16>(s[e], qa[1].x, qb[1].x, qa[1].y, qb[1].y, k1.x, k1.y);
        mma16816<T16>(s[e], qa[1].z, qb[1].z, qa[1].w, qb[1].w, k1.z, k1.w);
      }
      uint4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int vr = 2 * j + (e & 1) + (e >> 1) * 8;
        v[e] = *reinterpret_cast<const uint4*>(vb + vr * 128 + ((r ^ (vr & 7)) << 4));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < 2 * kRows; ++k) s[e][k] *= a.scale_log2;
      // a tile with rows outside the window, behind the end or before the
      // window's first: their scores go to -inf and their values to zero (a
      // row that nothing wrote may hold anything, NaN among it)
      const bool whole = pos0 + kTile <= n && (a.window <= 0 || pos0 >= n - a.window || pos0 + kTile <= a.sinks);
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (!visible(pos0 + 8 * e + 2 * j + k)) {
              s[e][k] = -INFINITY;
              s[e][k + 2] = -INFINITY;
              v[2 * e + k] = make_uint4(0, 0, 0, 0);
            }
      }
      float alpha[2] = {1.f, 1.f};
#pragma unroll
      for (int g = 0; g < kRows; ++g) {
        float mx = fmaxf(fmaxf(s[0][2 * g], s[0][2 * g + 1]), fmaxf(s[1][2 * g], s[1][2 * g + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(acc.m[g], mx);
        const float ms = mn == -INFINITY ? 0.f : mn;  // every score so far is -inf
        alpha[g] = acc.m[g] == mn ? 1.f : ex2_approx(acc.m[g] - ms);
        acc.m[g] = mn;
        acc.l[g] *= alpha[g];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            s[e][2 * g + k] = ex2_approx(s[e][2 * g + k] - ms + kShift<T16>);
            acc.l[g] += s[e][2 * g + k];
          }
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          acc.o[k][0] *= alpha[0];
          acc.o[k][1] *= alpha[0];
          acc.o[k][2] *= alpha[WIDE ? 1 : 0];
          acc.o[k][3] *= alpha[WIDE ? 1 : 0];
        }
      }
      uint32_t ph[2][2], pl[2][2];  // [position half][head half]
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int g = 0; g < kRows; ++g) split2<T16>(s[e][2 * g], s[e][2 * g + 1], ph[e][g], pl[e][g]);
      const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&v[0]);
      const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&v[1]);
      const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&v[2]);
      const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&v[3]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t sel = (k & 1) ? 0x7632u : 0x5410u;
        const uint32_t b0 = __byte_perm(v0[k >> 1], v1[k >> 1], sel);
        const uint32_t b1 = __byte_perm(v2[k >> 1], v3[k >> 1], sel);
        if constexpr (WIDE) {
          mma16816<T16>(acc.o[k], ph[0][0], ph[0][1], ph[1][0], ph[1][1], b0, b1);
          mma16816<T16>(acc.o[k], pl[0][0], pl[0][1], pl[1][0], pl[1][1], b0, b1);
        } else {
          mma16816<T16>(acc.o[k], ph[0][0], pl[0][0], ph[1][0], pl[1][0], b0, b1);
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
  for (int g = 0; g < 2; ++g) {  // sums over the four lanes of a row
    acc.l[g] += __shfl_xor_sync(0xffffffffu, acc.l[g], 1);
    acc.l[g] += __shfl_xor_sync(0xffffffffu, acc.l[g], 2);
  }
  if (!WIDE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc.o[i][0] += acc.o[i][2];
      acc.o[i][1] += acc.o[i][3];
    }
  }
  return true;
}

// The rows of one warp's result: dst[head][64], ml[head] = (m, l).
template <typename T16, bool WIDE>
__device__ __forceinline__ void put_piece(const Acc& acc, int heads, float* dst, float2* ml) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
#pragma unroll
  for (int g = 0; g < (WIDE ? 2 : 1); ++g) {
    const int hh = r + 8 * g;
    if (hh >= heads) continue;
    float* po = dst + hh * kHd + 16 * j;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      *reinterpret_cast<float4*>(po + 8 * e) =
          make_float4(acc.o[0][2 * g + e], acc.o[1][2 * g + e], acc.o[2][2 * g + e], acc.o[3][2 * g + e]);
      *reinterpret_cast<float4*>(po + 8 * e + 4) =
          make_float4(acc.o[4][2 * g + e], acc.o[5][2 * g + e], acc.o[6][2 * g + e], acc.o[7][2 * g + e]);
    }
    if (j == 0) ml[hh] = make_float2(acc.m[g] - kShift<T16>, acc.l[g]);
  }
}

// Adds a piece (its 4 values x, its m and l) to (acc, M, L).
__device__ __forceinline__ void merge(float4& acc, float& M, float& L, const float4& x, const float2& ml) {
  if (ml.y == 0.f) return;  // nothing in it but scores of -inf
  const float mn = fmaxf(M, ml.x);
  const float c0 = M == mn ? 1.f : ex2_approx(M - mn), c1 = ml.x == mn ? 1.f : ex2_approx(ml.x - mn);
  M = mn;
  L = L * c0 + ml.y * c1;
  acc.x = acc.x * c0 + x.x * c1;
  acc.y = acc.y * c0 + x.y * c1;
  acc.z = acc.z * c0 + x.z * c1;
  acc.w = acc.w * c0 + x.w * c1;
}

template <typename T16>
__device__ __forceinline__ Ring ring_of(const CUtensorMap* map, uint8_t* smem, uint64_t* bars, int warp) {
  Ring ring{map, smem + warp * kWarpBytes, bars + warp * kStages, 0, 0};
  if ((threadIdx.x & 31) == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(&ring.bar[s]), 1);
    fence_barrier_init();
  }
  __syncwarp();
  return ring;
}

// Work is cut into equal runs of tiles over all (sequence, key-value head,
// head block) items laid end to end, one run per warp, whatever the lengths
// are.  A warp that holds all tiles of an item writes its output; pieces of an
// item go to the workspace and a second kernel joins them.
//
// Measured (device time with the join; a copy reaches 6.69 TB/s): 64 sequences
// of 544 to 1087 positions, 12 heads, bf16: 33 us, 4.8 TB/s; 16 of 16K to 32K,
// 4 key-value heads for 16, fp16: 66 us, 5.9 TB/s; 128 under a window of 1024,
// 25 heads, bf16: 137 us, 6.1 TB/s.  What is left is the start (lengths, their
// sums, the table: loads that wait for one another, about 3 us) and the join
// (4.5 us).  The last case with other choices: fragments loaded from global
// memory into registers, 12 warps an SM, 169 us; three stages 143; five CTAs an
// SM 146; eight warps a CTA, or two, as four.
template <typename T16, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
    paged_attn(const __grid_constant__ CUtensorMap map, const PagedArgs<T16> a) {
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_bar[kWarps * kStages];
  __shared__ int s_sum[kWarps];
  uint8_t* s_tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  int* s_base = reinterpret_cast<int*>(s_tiles + kWarps * kWarpBytes);  // [n_seq + 1]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Ring ring = ring_of<T16>(&map, s_tiles, s_bar, warp);
  if (lane == 0) tma_prefetch_desc(&map);
  griddep_wait();
  const int items = a.n_kv * a.n_hb;
  // base[b] = tiles of all items of sequences before b
  int carry = 0;
  for (int b0 = 0; b0 < a.n_seq; b0 += kWarps * 32) {
    const int b = b0 + tid;
    int v = 0;
    if (b < a.n_seq) v = max(span_of(a, b, blockIdx.x == 0).nt, 0) * items;
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
  const int n_warps = gridDim.x * kWarps;
  const int run = max((total + n_warps - 1) / n_warps, WIDE ? 2 * kMinRun : kMinRun);
  if (blockIdx.x == 0) {
    for (int b = tid; b <= a.n_seq; b += kWarps * 32) a.plan[b] = s_base[b];
    if (tid == 0) a.plan[a.n_seq + 1] = run;
  }
  // neighbouring runs on different SMs, so that few runs use many SMs
  const int w = warp * gridDim.x + blockIdx.x;
  const long long t_first = static_cast<long long>(w) * run;
  if (t_first >= total) return;
  int t = static_cast<int>(t_first);
  const int t_end = static_cast<int>(min(t_first + run, static_cast<long long>(total)));
  const int r = lane >> 2, j = lane & 3;

  while (t < t_end) {
    int lo = 0, hi = a.n_seq;  // last b with base[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_base[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const Span sp = span_of(a, lo, false);
    const int item = (t - s_base[lo]) / sp.nt;
    const int j0 = (t - s_base[lo]) - item * sp.nt;  // first tile of this piece within the item
    const int cnt = min(sp.nt - j0, t_end - t);
    const Item<T16> x = item_of(a, lo, item, sp);
    Acc acc;
    if (!attend<T16, WIDE>(a, x, j0, 1, cnt, ring, acc)) return;
    // the join may come now; earlier, its CTAs, waiting in the places of ours
    // that are through, cost a window case of 128 sequences 169 us instead of 137
    if (t + cnt >= t_end) griddep_launch_dependents();
    if (cnt == sp.nt) {
#pragma unroll
      for (int g = 0; g < (WIDE ? 2 : 1); ++g) {
        const int hh = r + 8 * g;
        if (hh >= x.heads) continue;
        const float l = acc.l[g], inv = l == 0.f ? 0.f : 1.f / l;
        T16* orow = a.out + x.b * a.ldo + static_cast<long long>(x.head0 + hh) * kHd + 16 * j;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint4 u;
          u.x = Type16<T16>::pack2(acc.o[0][2 * g + e] * inv, acc.o[1][2 * g + e] * inv);
          u.y = Type16<T16>::pack2(acc.o[2][2 * g + e] * inv, acc.o[3][2 * g + e] * inv);
          u.z = Type16<T16>::pack2(acc.o[4][2 * g + e] * inv, acc.o[5][2 * g + e] * inv);
          u.w = Type16<T16>::pack2(acc.o[6][2 * g + e] * inv, acc.o[7][2 * g + e] * inv);
          *reinterpret_cast<uint4*>(orow + 8 * e) = u;
        }
        if (a.lse && j == 0)
          a.lse[static_cast<long long>(x.b) * a.H + x.head0 + hh] = acc.m[g] - kShift<T16> + log2f(l);
      }
    } else {
      const long long slot = 2ll * w + (t == static_cast<int>(t_first) ? 0 : 1);
      put_piece<T16, WIDE>(acc, x.heads, a.part_o + slot * a.HB * kHd, a.part_ml + slot * a.HB);
    }
    t += cnt;
  }
}

// The pieces of an item: warps w0 .. w1 of paged_attn hold one each (w0 > w1:
// no positions).  False if there is nothing to join.
template <typename T16>
__device__ __forceinline__ bool pieces_of(const PagedArgs<T16>& a, int b, int item, const Span& sp, int& w0, int& w1,
                                          bool& second) {
  const int run = a.plan[a.n_seq + 1];
  const int s = a.plan[b] + item * sp.nt;
  w0 = s / run;
  w1 = sp.nt > 0 ? (s + sp.nt - 1) / run : w0 - 1;
  second = s != w0 * run;  // the item began within the first warp's run: its second slot
  return w0 != w1;         // else that warp wrote the output
}

// Four dimensions of one head over the pieces w, w + ways, ..., kAhead of them
// on their way at a time.
constexpr int kAhead = 4;
template <typename T16>
__device__ __forceinline__ void gather(const PagedArgs<T16>& a, int w, int ways, int w0, int w1, bool second, int hh,
                                       int d4, float4& acc, float& M, float& L) {
  for (; w <= w1; w += kAhead * ways) {
    float4 x[kAhead];
    float2 ml[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int wu = w + u * ways;
      ml[u] = make_float2(-INFINITY, 0.f);
      if (wu <= w1) {
        const long long at = (2ll * wu + (wu == w0 && second ? 1 : 0)) * a.HB + hh;
        ml[u] = a.part_ml[at];
        x[u] = *reinterpret_cast<const float4*>(a.part_o + at * kHd + 4 * d4);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) merge(acc, M, L, x[u], ml[u]);
  }
}

template <typename T16>
__device__ __forceinline__ void put_joined(const PagedArgs<T16>& a, int b, int head, int d4, const float4& acc, float M,
                                           float L) {
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint2 v;
  v.x = Type16<T16>::pack2(acc.x * inv, acc.y * inv);
  v.y = Type16<T16>::pack2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(a.out + b * a.ldo + static_cast<long long>(head) * kHd + 4 * d4) = v;
  if (a.lse && d4 == 0) a.lse[static_cast<long long>(b) * a.H + head] = M + log2f(L);
}

// Joins the pieces of items that several warps shared, in a fixed order, and
// writes zeros (log-sum-exp -inf) for a sequence with nothing visible.
//
// With many items each has few pieces: one warp per item, 16 lanes for a
// head's 64 dimensions, two heads at a time or one head's pieces in two halves.
constexpr int kJoinThreads = 128;
template <typename T16>
__global__ void __launch_bounds__(kJoinThreads) paged_join_many(const PagedArgs<T16> a) {
  const int items = a.n_kv * a.n_hb, lane = threadIdx.x & 31;
  const int k = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int b = k / items, item = k - b * items;
  // the lengths are older than the kernel before, which has waited for them
  Span sp{0, 0, 0, -1};
  if (b < a.n_seq) sp = span_of(a, b, false);
  griddep_wait();
  griddep_launch_dependents();
  int w0, w1;
  bool second;
  if (sp.nt < 0 || !pieces_of(a, b, item, sp, w0, w1, second)) return;
  const Item<T16> x = item_of(a, b, item, sp);
  const int half = lane >> 4, d4 = lane & 15;
  const bool one = x.heads == 1;
  for (int h0 = 0; h0 < x.heads; h0 += 2) {
    const int hh = one ? 0 : h0 + half;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (hh < x.heads) gather(a, one ? w0 + half : w0, one ? 2 : 1, w0, w1, second, hh, d4, acc, M, L);
    if (one) {
      const float4 o = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, 16), __shfl_xor_sync(0xffffffffu, acc.y, 16),
                                   __shfl_xor_sync(0xffffffffu, acc.z, 16), __shfl_xor_sync(0xffffffffu, acc.w, 16));
      const float2 ml = make_float2(__shfl_xor_sync(0xffffffffu, M, 16), __shfl_xor_sync(0xffffffffu, L, 16));
      merge(acc, M, L, o, ml);
    }
    if (one ? half == 0 : hh < x.heads) put_joined(a, b, x.head0 + hh, d4, acc, M, L);
  }
}

// With few items each has many pieces: one CTA for `width` heads of an item
// (blockIdx.y: which), side by side; the groups of threads that are left take
// every ways-th piece.
constexpr int kJoinFewThreads = 512;
template <typename T16>
__global__ void __launch_bounds__(kJoinFewThreads) paged_join_few(const PagedArgs<T16> a, int width) {
  __shared__ float4 s_o[kJoinFewThreads];
  __shared__ float2 s_ml[kJoinFewThreads];
  const int items = a.n_kv * a.n_hb;
  const int b = blockIdx.x / items, item = blockIdx.x - b * items;
  const Span sp = span_of(a, b, false);
  griddep_wait();
  griddep_launch_dependents();
  int w0, w1;
  bool second;
  if (sp.nt < 0 || !pieces_of(a, b, item, sp, w0, w1, second)) return;
  const Item<T16> x = item_of(a, b, item, sp);
  const int ways = kJoinFewThreads / 16 / width;
  const int tid = threadIdx.x, d4 = tid & 15, way = (tid >> 4) / width;
  const int hh = blockIdx.y * width + (tid >> 4) % width;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (hh < x.heads) gather(a, w0 + way, ways, w0, w1, second, hh, d4, acc, M, L);
  s_o[tid] = acc;
  s_ml[tid] = make_float2(M, L);
  // pairwise, in an order that the number of threads alone gives
  for (int k = ways >> 1; k > 0; k >>= 1) {
    __syncthreads();
    if (way < k) {
      merge(acc, M, L, s_o[tid + 16 * width * k], s_ml[tid + 16 * width * k]);
      s_o[tid] = acc;
      s_ml[tid] = make_float2(M, L);
    }
  }
  if (way == 0 && hh < x.heads) put_joined(a, b, x.head0 + hh, d4, acc, M, L);
}

// The same work with one CTA per item and nothing to join afterwards: 16 warps
// take every 16th tile and meet in shared memory.  For few items of bounded
// length (one or a few conversations on a small model), where a second launch
// would cost more than spreading an item over several SMs saves: one sequence
// of 777 positions at 12 heads takes 6.9 us, and 9.2 in runs that are joined.
// The host does not know the lengths: what counts is the table's width (or the
// window), so a conversation in a table of more than 2048 positions is joined.
constexpr int kSoloWarps = 16;
constexpr int kSoloTiles = 128;  // 2048 positions
template <typename T16, bool WIDE>
__global__ void __launch_bounds__(kSoloWarps * 32, 1)
    paged_attn_solo(const __grid_constant__ CUtensorMap map, const PagedArgs<T16> a) {
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_bar[kSoloWarps * kStages];
  __shared__ float2 s_ml[kSoloWarps * 16];
  uint8_t* s_tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5;
  Ring ring = ring_of<T16>(&map, s_tiles, s_bar, warp);
  if (tid == 0) tma_prefetch_desc(&map);
  griddep_wait();
  griddep_launch_dependents();
  const int items = a.n_kv * a.n_hb;
  const int b = blockIdx.x / items, item = blockIdx.x - b * items;
  const Span sp = span_of(a, b, item == 0 && tid == 0);
  if (sp.nt < 0) return;
  const Item<T16> x = item_of(a, b, item, sp);
  const int cnt = sp.nt > warp ? (sp.nt - warp + kSoloWarps - 1) / kSoloWarps : 0;
  Acc acc;
  // the ring's own bytes take the warp's result once its tiles are through: at
  // most 16 heads of 256 bytes
  float* mine = reinterpret_cast<float*>(ring.buf);
  if (cnt > 0) {
    if (attend<T16, WIDE>(a, x, warp, kSoloWarps, cnt, ring, acc)) {
      __syncwarp();
      put_piece<T16, WIDE>(acc, x.heads, mine, s_ml + warp * 16);
    } else if ((tid & 31) < 16) {
      s_ml[warp * 16 + (tid & 31)] = make_float2(-INFINITY, 0.f);
    }
  }
  __syncthreads();
  const int pieces = min(sp.nt, kSoloWarps);
  for (int k = tid; k < x.heads * 16; k += kSoloWarps * 32) {
    const int hh = k >> 4, d4 = k & 15;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < pieces; ++w)
      merge(o, M, L, *reinterpret_cast<const float4*>(s_tiles + w * kWarpBytes + (hh * kHd + 4 * d4) * 4),
            s_ml[w * 16 + hh]);
    put_joined(a, b, x.head0 + hh, d4, o, M, L);
  }
}

// Query heads of one key-value head in blocks of at most 16 (rows of the A
// operand), as even as they come.
int head_blocks(int group) { return (group + 15) / 16; }

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
int max_warps() { return num_sms() * kCtasPerSm * kWarps; }

template <typename T16>
cudaError_t launch_t(const gpt2_paged_cache* c, int layer, const void* q, int64_t ldq, const void* k_new,
                     const void* v_new, int64_t ldkv, void* out, int64_t ldo, float* lse, int n_head,
                     float score_scale, int window, int sinks, void* ws, cudaStream_t s) {
  const int sms = num_sms();
  PagedArgs<T16> a;
  a.q = static_cast<const T16*>(q);
  a.k_new = static_cast<const T16*>(k_new);
  a.v_new = static_cast<const T16*>(v_new);
  a.out = static_cast<T16*>(out);
  a.lse = lse;
  const long long layer_elems = 2ll * c->n_kv_head * c->page_size * kHd;
  a.pages = static_cast<T16*>(c->pages) + layer * layer_elems;
  a.page_rows = c->n_layer * 2 * c->n_kv_head * c->page_size;
  a.row0 = layer * 2 * c->n_kv_head * c->page_size;
  a.table = c->table;
  a.lens = c->lens;
  a.refs = c->refs;
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
  a.n_hb = head_blocks(a.group);
  a.HB = (a.group + a.n_hb - 1) / a.n_hb;
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = score_scale * 1.4426950408889634f;
  char* base = static_cast<char*>(ws);
  a.plan = reinterpret_cast<int*>(base);
  base += align256((static_cast<size_t>(c->n_seq) + 2) * 4);
  a.part_ml = reinterpret_cast<float2*>(base);
  base += align256(2ull * sms * kCtasPerSm * kWarps * a.HB * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(base);
  // the pool as one [rows, 64] matrix
  const uint64_t rows = static_cast<uint64_t>(c->n_pages) * a.page_rows;
  CUtensorMap map;
  if (!encode_tma_2d(&map, Type16<T16>::kTma, c->pages, kHd, rows, kHd * 2, kHd, kTile)) return cudaErrorInvalidValue;
  const bool wide = a.HB > 8;
  const long long items = static_cast<long long>(c->n_seq) * a.n_kv * a.n_hb;
  // positions that a query can see: of the window, of the sinks, and what
  // shares a tile with either
  long long most = static_cast<long long>(c->max_pages) * c->page_size;
  if (window > 0) most = std::min(most, static_cast<long long>(window) + sinks + 3 * kTile);
  const bool solo = items <= sms && most <= kSoloTiles * kTile;
  const int smem = solo ? kSoloWarps * kWarpBytes + 1024 : kWarps * kWarpBytes + 1024 + (c->n_seq + 1) * 4;
  auto kern = solo ? (wide ? paged_attn_solo<T16, true> : paged_attn_solo<T16, false>)
                   : (wide ? paged_attn<T16, true> : paged_attn<T16, false>);
  static int configured[4][64] = {{0}};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int& done = configured[2 * solo + wide][dev];
  if (!done) {
    cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
        solo ? kSoloWarps * kWarpBytes + 1024 : kWarps * kWarpBytes + 1024 + (kMaxPagedSeqs + 1) * 4);
    if (e != cudaSuccess) return e;
    // the joins use little shared memory but leave the SMs split as paged_attn
    // has them: between two splits an SM has to run empty
    e = cudaFuncSetAttribute(paged_join_many<T16>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(paged_join_few<T16>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    done = 1;
  }
  if (solo) return launch_pdl(kern, static_cast<unsigned>(items), kSoloWarps * 32, smem, s, 0, map, a);
  cudaError_t e = launch_pdl(kern, sms * kCtasPerSm, kWarps * 32, smem, s, 0, map, a);
  if (e != cudaSuccess) return e;
  if (items > sms) {
    const unsigned joins = static_cast<unsigned>((items + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
    return launch_pdl(paged_join_many<T16>, joins, kJoinThreads, 0, s, 0, a);
  }
  int width = 1;  // as many CTAs as there are places for
  while (width < 8 && items * ((a.HB + width - 1) / width) > 2 * sms) width *= 2;
  return launch_pdl(paged_join_few<T16>, dim3(static_cast<unsigned>(items), (a.HB + width - 1) / width),
                    kJoinFewThreads, 0, s, 0, a, width);
}

}  // namespace

size_t attention_paged_workspace(const gpt2_paged_cache* c, int n_head) {
  const int group = n_head / c->n_kv_head, n_hb = head_blocks(group), HB = (group + n_hb - 1) / n_hb;
  const size_t slots = 2ull * max_warps() * HB;
  return align256((static_cast<size_t>(c->n_seq) + 2) * 4) + align256(slots * sizeof(float2)) +
         align256(slots * kHd * 4);
}

bool attention_paged_fits(const gpt2_paged_cache* c, int n_head) {
  // rows of the pool are TMA coordinates, and tiles of all items are counted,
  // in 32 bits, the latter with room for one run more
  const int group = n_head / c->n_kv_head;
  if (static_cast<double>(c->n_pages) * c->n_layer * 2 * c->n_kv_head * c->page_size >= 2147483648.0) return false;
  return static_cast<long long>(c->n_seq) * c->n_kv_head * head_blocks(group) *
             (static_cast<long long>(c->max_pages) * c->page_size / kTile) <
         (1ll << 30);
}

cudaError_t launch_attention_paged(const gpt2_paged_cache* c, int layer, const void* q, int64_t ldq,
                                   const void* k_new, const void* v_new, int64_t ldkv, void* out, int64_t ldo,
                                   float* lse, int n_head, float score_scale, int window, int sinks, void* ws,
                                   cudaStream_t s) {
  return c->dtype == GPT2_F16 ? launch_t<__half>(c, layer, q, ldq, k_new, v_new, ldkv, out, ldo, lse, n_head,
                                                 score_scale, window, sinks, ws, s)
                              : launch_t<__nv_bfloat16>(c, layer, q, ldq, k_new, v_new, ldkv, out, ldo, lse, n_head,
                                                        score_scale, window, sinks, ws, s);
}

}  // namespace gpt2
