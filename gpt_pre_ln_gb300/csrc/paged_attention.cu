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
// Every visible key and value row is read once (256 bytes a position and
// key-value head) and takes 4 * 64 flop per query head: at most 16 flop a byte
// with 16 heads to a key-value head, far under what the tensor cores need to
// be the limit, so the kernel is bound by HBM bandwidth and its layout serves
// the loads.  The products run as mma.sync m16n8k16 on fragments loaded from
// global memory straight into registers: no shared memory, no barriers, no
// waits, and nothing to gain from tcgen05, whose operands would have to pass
// through shared memory first.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace gpt2 {

namespace {

constexpr int kHd = 64;
constexpr int kTile = 16;    // positions per tile; page sizes are multiples of it
constexpr int kWarps = 4;    // warps per CTA, independent of one another
constexpr int kCtasPerSm = 3;

template <typename T16>
struct PagedArgs {
  const T16* q;
  const T16* k_new;  // null: the query attends over the cached positions only
  const T16* v_new;
  T16* out;
  float* lse;  // nullable, [n_seq, H]
  T16* pages;  // the layer's part of page 0
  const int32_t* table;
  const int32_t* lens;
  int* plan;       // base[n_seq + 1], then tiles per warp
  float* part_o;   // [2 * warps, HB, 64]
  float2* part_ml;  // [2 * warps, HB]: running maximum (log2 units) and sum
  unsigned* err;
  long long ldq, ldkv, ldo, page_stride;
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
  const int len = a.lens[b];
  const int n = len + (a.k_new ? 1 : 0);
  Span s{n, 0, 0, -1};
  if (len < 0) return s;
  if (n > a.max_pages * a.page_size) {
    if (record) record_error(a.err, kErrRange, kSitePagedLength);
    return s;
  }
  const int te = (n + kTile - 1) / kTile;
  if (a.window > 0 && n > a.window) {
    const int first = n - a.window;
    s.tw = first / kTile;
    s.ts = min((min(a.sinks, first) + kTile - 1) / kTile, s.tw);
  }
  s.nt = s.ts + te - s.tw;
  return s;
}

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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

// One tile's keys and values in a warp's registers.  Lane (r = lane / 4,
// j = lane % 4) holds of key rows r and r + 8 the dimensions 8j..8j+7 and
// 32+8j..32+8j+7, and of value rows 2j, 2j+1, 2j+8, 2j+9 the dimensions
// 8r..8r+7, each 16 bytes.  The sums over dimensions and the order of output
// dimensions are free, so these are the B fragments of both products as they
// come: keys with the contraction index permuted alike in q, values with
// output column r of product t standing for dimension 8r + t.
struct TileRegs {
  uint4 k[2][2];
  uint4 v[4];
  int pos0;  // first position, or -1: the tile's page is not there
};

// (p rounded, what that lost) in 16 bits, so that their sum carries p to 16
// bits (bf16) or 22 bits (fp16).
template <typename T16>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = Type16<T16>::pack2(x, y);
  const float2 h = Type16<T16>::unpack2(hi);
  lo = Type16<T16>::pack2(x - h.x, y - h.y);
}

// Work is cut into equal runs of tiles over all (sequence, key-value head,
// head block) items laid end to end, one run per warp, whatever the lengths
// are.  A warp that holds all tiles of an item writes its output; pieces of an
// item go to the workspace and paged_join adds them up.
//
// WIDE: 9 to 16 query heads per block fill the 16 rows of the A operand; the
// rounding remainder of p then takes a second product.  Up to 8 heads leave
// rows 8..15 free and the remainder rides there.
template <typename T16, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) paged_attn(const PagedArgs<T16> a) {
  extern __shared__ int s_base[];  // [n_seq + 1]
  __shared__ int s_sum[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  const int run = max((total + n_warps - 1) / n_warps, 1);
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
  // fp16 probabilities are carried 2^12 times larger: their smallest step is
  // then 2^-36 of the row's largest and not 2^-24
  constexpr float kShift = std::is_same<T16, __half>::value ? 12.f : 0.f;

  while (t < t_end) {
    int lo = 0, hi = a.n_seq;  // last b with base[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_base[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const int b = lo;
    const Span sp = span_of(a, b, false);
    const int item = (t - s_base[b]) / sp.nt;
    const int j0 = (t - s_base[b]) - item * sp.nt;  // first tile of this piece within the item
    const int cnt = min(sp.nt - j0, t_end - t);
    const int kvh = item / a.n_hb, hb = item - kvh * a.n_hb;
    const int head0 = kvh * a.group + hb * a.HB;
    const int heads = min(a.HB, a.group - hb * a.HB);
    const int pos_new = a.k_new ? sp.n - 1 : -1;
    const T16* kn = a.k_new + b * a.ldkv + kvh * kHd;
    const T16* vn = a.v_new + b * a.ldkv + kvh * kHd;
    const int32_t* trow = a.table + static_cast<long long>(b) * a.max_pages;

    // q fragments: rows r (and r + 8 when WIDE)
    uint4 qa[2] = {}, qb[2] = {};
    {
      const T16* qr = a.q + b * a.ldq + static_cast<long long>(head0 + r) * kHd + 8 * j;
      if (r < heads) {
        qa[0] = load16(qr);
        qa[1] = load16(qr + 32);
      }
      if (WIDE && r + 8 < heads) {
        qb[0] = load16(qr + 8 * kHd);
        qb[1] = load16(qr + 8 * kHd + 32);
      }
    }
    float o[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    int pages32 = -1;  // lane i: the page of tile (tile index & ~31) + i of this piece
    auto tile_no = [&](int i) { return i < sp.ts ? i : sp.tw + (i - sp.ts); };
    auto fetch = [&](int i, TileRegs& x) {  // i: tile within the piece
      if ((i & 31) == 0) {
        const int ii = j0 + i + lane;
        pages32 = i + lane < cnt ? trow[tile_no(ii) * kTile / a.page_size] : -1;
      }
      const int page = __shfl_sync(0xffffffffu, pages32, i & 31);
      const int pos0 = tile_no(j0 + i) * kTile;
      if (page < 0 || page >= a.n_pages) {
        if (lane == 0) record_error(a.err, kErrRange, kSitePagedPage);
        x.pos0 = -1;
        return;
      }
      x.pos0 = pos0;
      const T16* kb = a.pages + page * a.page_stride +
                      (static_cast<long long>(kvh) * a.page_size + pos0 % a.page_size) * kHd;
      const T16* vb = kb + static_cast<long long>(a.n_kv) * a.page_size * kHd;
      const T16* kr[2] = {kb + r * kHd, kb + (r + 8) * kHd};
      const T16* vr[4] = {vb + (2 * j) * kHd, vb + (2 * j + 1) * kHd, vb + (2 * j + 8) * kHd,
                          vb + (2 * j + 9) * kHd};
      const int at = pos_new - pos0;  // the new token's row in this tile
      if (pos_new >= 0 && at < kTile && at >= 0) {
        // its key and value come from the caller's rows and go to the cache
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (at == r + 8 * e) kr[e] = kn;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at == 2 * j + (e & 1) + (e >> 1) * 8) vr[e] = vn;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x.k[e][0] = load16(kr[e] + 8 * j);
        x.k[e][1] = load16(kr[e] + 32 + 8 * j);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x.v[e] = load16(vr[e] + 8 * r);
      if (pos_new >= 0 && at < kTile && at >= 0 && hb == 0) {
        T16* kc = const_cast<T16*>(kb) + at * kHd;
        T16* vc = const_cast<T16*>(vb) + at * kHd;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (at == r + 8 * e) {
            *reinterpret_cast<uint4*>(kc + 8 * j) = x.k[e][0];
            *reinterpret_cast<uint4*>(kc + 32 + 8 * j) = x.k[e][1];
          }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at == 2 * j + (e & 1) + (e >> 1) * 8) *reinterpret_cast<uint4*>(vc + 8 * r) = x.v[e];
      }
    };
    auto visible = [&](int p) {
      return p < sp.n && (a.window <= 0 || p >= sp.n - a.window || p < a.sinks);
    };
    auto consume = [&](TileRegs& x) {
      if (x.pos0 < 0) return;
      float s[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[e][0] = s[e][1] = s[e][2] = s[e][3] = 0.f;
        mma16816<T16>(s[e], qa[0].x, qb[0].x, qa[0].y, qb[0].y, x.k[e][0].x, x.k[e][0].y);
        mma16816<T16>(s[e], qa[0].z, qb[0].z, qa[0].w, qb[0].w, x.k[e][0].z, x.k[e][0].w);
        mma16816<T16>(s[e], qa[1].x, qb[1].x, qa[1].y, qb[1].y, x.k[e][1].x, x.k[e][1].y);
        mma16816<T16>(s[e], qa[1].z, qb[1].z, qa[1].w, qb[1].w, x.k[e][1].z, x.k[e][1].w);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[e][i] *= a.scale_log2;
      // a tile with rows outside the window, behind the end or before the
      // window's first: their scores go to -inf and their values to zero (a
      // row that nothing wrote may hold anything, NaN among it)
      const bool whole = x.pos0 + kTile <= sp.n &&
                         (a.window <= 0 || x.pos0 >= sp.n - a.window || x.pos0 + kTile <= a.sinks);
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (!visible(x.pos0 + 8 * e + 2 * j + i)) {
              s[e][i] = -INFINITY;
              s[e][i + 2] = -INFINITY;
              x.v[2 * e + i] = make_uint4(0, 0, 0, 0);
            }
      }
      constexpr int kRows = WIDE ? 2 : 1;
      float alpha[2] = {1.f, 1.f};
#pragma unroll
      for (int g = 0; g < kRows; ++g) {
        float mx = fmaxf(fmaxf(s[0][2 * g], s[0][2 * g + 1]), fmaxf(s[1][2 * g], s[1][2 * g + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[g], mx);
        const float ms = mn == -INFINITY ? 0.f : mn;  // every score so far is -inf
        alpha[g] = m[g] == mn ? 1.f : ex2_approx(m[g] - ms);
        m[g] = mn;
        l[g] *= alpha[g];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            s[e][2 * g + i] = ex2_approx(s[e][2 * g + i] - ms + kShift);
            l[g] += s[e][2 * g + i];
          }
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          o[i][2] *= alpha[WIDE ? 1 : 0];
          o[i][3] *= alpha[WIDE ? 1 : 0];
        }
      }
      uint32_t ph[2][2], pl[2][2];  // [position half][head half]
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int g = 0; g < kRows; ++g) split2<T16>(s[e][2 * g], s[e][2 * g + 1], ph[e][g], pl[e][g]);
      const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&x.v[0]);
      const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&x.v[1]);
      const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&x.v[2]);
      const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&x.v[3]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
        const uint32_t b0 = __byte_perm(v0[i >> 1], v1[i >> 1], sel);
        const uint32_t b1 = __byte_perm(v2[i >> 1], v3[i >> 1], sel);
        if constexpr (WIDE) {
          mma16816<T16>(o[i], ph[0][0], ph[0][1], ph[1][0], ph[1][1], b0, b1);
          mma16816<T16>(o[i], pl[0][0], pl[0][1], pl[1][0], pl[1][1], b0, b1);
        } else {
          mma16816<T16>(o[i], ph[0][0], pl[0][0], ph[1][0], pl[1][0], b0, b1);
        }
      }
    };

    TileRegs x0, x1;
    fetch(0, x0);
    for (int i = 0; i < cnt; i += 2) {
      if (i + 1 < cnt) fetch(i + 1, x1);
      consume(x0);
      if (i + 2 < cnt) fetch(i + 2, x0);
      if (i + 1 < cnt) consume(x1);
    }

    // sums over the four lanes of a row
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      l[g] += __shfl_xor_sync(0xffffffffu, l[g], 1);
      l[g] += __shfl_xor_sync(0xffffffffu, l[g], 2);
    }
    if (!WIDE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i][0] += o[i][2];
        o[i][1] += o[i][3];
      }
    }
    const bool complete = cnt == sp.nt;
    const int slot = 2 * w + (t == static_cast<int>(t_first) ? 0 : 1);
    // lane (r, j) holds dimensions 16j + i and 16j + 8 + i of heads r (and r + 8)
#pragma unroll
    for (int g = 0; g < (WIDE ? 2 : 1); ++g) {
      const int hh = r + 8 * g;
      if (hh < heads) {
        if (complete) {
          const float inv = l[g] > 0.f ? 1.f / l[g] : 0.f;
          T16* orow = a.out + b * a.ldo + static_cast<long long>(head0 + hh) * kHd + 16 * j;
          uint4 lo4, hi4;
          lo4.x = Type16<T16>::pack2(o[0][2 * g] * inv, o[1][2 * g] * inv);
          lo4.y = Type16<T16>::pack2(o[2][2 * g] * inv, o[3][2 * g] * inv);
          lo4.z = Type16<T16>::pack2(o[4][2 * g] * inv, o[5][2 * g] * inv);
          lo4.w = Type16<T16>::pack2(o[6][2 * g] * inv, o[7][2 * g] * inv);
          hi4.x = Type16<T16>::pack2(o[0][2 * g + 1] * inv, o[1][2 * g + 1] * inv);
          hi4.y = Type16<T16>::pack2(o[2][2 * g + 1] * inv, o[3][2 * g + 1] * inv);
          hi4.z = Type16<T16>::pack2(o[4][2 * g + 1] * inv, o[5][2 * g + 1] * inv);
          hi4.w = Type16<T16>::pack2(o[6][2 * g + 1] * inv, o[7][2 * g + 1] * inv);
          *reinterpret_cast<uint4*>(orow) = lo4;
          *reinterpret_cast<uint4*>(orow + 8) = hi4;
          if (a.lse && j == 0) a.lse[static_cast<long long>(b) * a.H + head0 + hh] = m[g] - kShift + log2f(l[g]);
        } else {
          float* po = a.part_o + (static_cast<long long>(slot) * a.HB + hh) * kHd + 16 * j;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            *reinterpret_cast<float4*>(po + 8 * e) =
                make_float4(o[0][2 * g + e], o[1][2 * g + e], o[2][2 * g + e], o[3][2 * g + e]);
            *reinterpret_cast<float4*>(po + 8 * e + 4) =
                make_float4(o[4][2 * g + e], o[5][2 * g + e], o[6][2 * g + e], o[7][2 * g + e]);
          }
          if (j == 0) a.part_ml[static_cast<long long>(slot) * a.HB + hh] = make_float2(m[g] - kShift, l[g]);
        }
      }
    }
    t += cnt;
  }
}

// Joins the pieces of items that several warps shared, in the order of their
// positions, and writes zeros (log-sum-exp -inf) for a sequence with nothing
// visible.  One CTA per item; 16 threads hold one head's 64 dimensions, and
// the threads left over take every n-th piece of it.
constexpr int kJoinThreads = 128;
template <typename T16>
__global__ void __launch_bounds__(kJoinThreads) paged_join(const PagedArgs<T16> a) {
  __shared__ float4 s_o[kJoinThreads];
  __shared__ float2 s_ml[kJoinThreads];
  griddep_wait();
  griddep_launch_dependents();
  const int items = a.n_kv * a.n_hb;
  const int b = blockIdx.x / items, item = blockIdx.x - b * items;
  const Span sp = span_of(a, b, false);
  if (sp.nt < 0) return;
  const int run = a.plan[a.n_seq + 1];
  const int s = a.plan[b] + item * sp.nt, e = s + sp.nt;
  const int w0 = s / run, w1 = sp.nt > 0 ? (e - 1) / run : w0 - 1;
  if (w0 == w1) return;  // its warp wrote the output
  const int kvh = item / a.n_hb, hb = item - kvh * a.n_hb;
  const int head0 = kvh * a.group + hb * a.HB;
  const int heads = min(a.HB, a.group - hb * a.HB);
  const int tid = threadIdx.x, d4 = tid & 15;
  int width = 1;  // heads side by side: a power of two, at most 8
  while (width < heads && width < kJoinThreads / 16) width *= 2;
  const int ways = kJoinThreads / 16 / width;
  for (int h0 = 0; h0 < heads; h0 += width) {
    const int hh = h0 + (tid >> 4) % width, way = (tid >> 4) / width;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (hh < heads) {
      for (int w = w0 + way; w <= w1; w += ways) {
        const long long at = (2ll * w + (w == w0 && s != w * run ? 1 : 0)) * a.HB + hh;
        const float2 ml = a.part_ml[at];
        const float4 x = *reinterpret_cast<const float4*>(a.part_o + at * kHd + 4 * d4);
        if (!(ml.y > 0.f)) {
          if (ml.y == 0.f) continue;  // nothing in this piece but scores of -inf
        }
        const float mn = fmaxf(M, ml.x);
        const float c0 = M == mn ? 1.f : ex2_approx(M - mn), c1 = ml.x == mn ? 1.f : ex2_approx(ml.x - mn);
        M = mn;
        L = L * c0 + ml.y * c1;
        acc.x = acc.x * c0 + x.x * c1;
        acc.y = acc.y * c0 + x.y * c1;
        acc.z = acc.z * c0 + x.z * c1;
        acc.w = acc.w * c0 + x.w * c1;
      }
    }
    s_o[tid] = acc;
    s_ml[tid] = make_float2(M, L);
    __syncthreads();
    if (way == 0 && hh < heads) {
      for (int k = 1; k < ways; ++k) {
        const float2 ml = s_ml[tid + 16 * width * k];
        const float4 x = s_o[tid + 16 * width * k];
        if (ml.y == 0.f) continue;
        const float mn = fmaxf(M, ml.x);
        const float c0 = M == mn ? 1.f : ex2_approx(M - mn), c1 = ml.x == mn ? 1.f : ex2_approx(ml.x - mn);
        M = mn;
        L = L * c0 + ml.y * c1;
        acc.x = acc.x * c0 + x.x * c1;
        acc.y = acc.y * c0 + x.y * c1;
        acc.z = acc.z * c0 + x.z * c1;
        acc.w = acc.w * c0 + x.w * c1;
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      uint2 v;
      v.x = Type16<T16>::pack2(acc.x * inv, acc.y * inv);
      v.y = Type16<T16>::pack2(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(a.out + b * a.ldo + static_cast<long long>(head0 + hh) * kHd + 4 * d4) = v;
      if (a.lse && d4 == 0) a.lse[static_cast<long long>(b) * a.H + head0 + hh] = M + log2f(L);
    }
    __syncthreads();
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
  PagedArgs<T16> a;
  a.q = static_cast<const T16*>(q);
  a.k_new = static_cast<const T16*>(k_new);
  a.v_new = static_cast<const T16*>(v_new);
  a.out = static_cast<T16*>(out);
  a.lse = lse;
  const long long layer_elems = 2ll * c->n_kv_head * c->page_size * kHd;
  a.pages = static_cast<T16*>(c->pages) + layer * layer_elems;
  a.page_stride = layer_elems * c->n_layer;
  a.table = c->table;
  a.lens = c->lens;
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
  base += align256(2ull * max_warps() * a.HB * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(base);
  const unsigned grid = static_cast<unsigned>(num_sms() * kCtasPerSm);
  const size_t smem = (static_cast<size_t>(c->n_seq) + 1) * 4;
  cudaError_t e = a.HB > 8 ? launch_pdl(paged_attn<T16, true>, grid, kWarps * 32, smem, s, 0, a)
                           : launch_pdl(paged_attn<T16, false>, grid, kWarps * 32, smem, s, 0, a);
  if (e != cudaSuccess) return e;
  const unsigned joins = static_cast<unsigned>(c->n_seq) * a.n_kv * a.n_hb;
  return launch_pdl(paged_join<T16>, joins, kJoinThreads, 0, s, 0, a);
}

}  // namespace

size_t attention_paged_workspace(const gpt2_paged_cache* c, int n_head) {
  const int group = n_head / c->n_kv_head, n_hb = head_blocks(group), HB = (group + n_hb - 1) / n_hb;
  const size_t slots = 2ull * max_warps() * HB;
  return align256((static_cast<size_t>(c->n_seq) + 2) * 4) + align256(slots * sizeof(float2)) +
         align256(slots * kHd * 4);
}

bool attention_paged_fits(const gpt2_paged_cache* c, int n_head) {
  // tiles of all items are counted in 32 bits, with room for one run more
  const int group = n_head / c->n_kv_head;
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
