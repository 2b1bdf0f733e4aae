// Scores from stored logits: log probabilities of given tokens, the entropy
// of each row's distribution and its most likely alternatives.
//
//   m = max z, S = sum e^(z - m), lse = m + log S,
//   log p(v) = (z_v - m) - log S, H = log S - sum e^(z - m) (z - m) / S.
//
// Reading the logits once is all that has to move; the arithmetic (a handful
// of operations and one exponential per logit) is of the same order as the
// memory time.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace gpt2 {

namespace {

struct Cand {
  float v;
  int i;
};
// the order of the alternatives: larger value first, lower index on ties
__device__ __forceinline__ bool ahead(const Cand& a, const Cand& b) { return a.v > b.v || (a.v == b.v && a.i < b.i); }

// 16 bytes of logits as pairs of floats; as packed 16-bit pairs for maxima.
template <typename T>
struct Row16 {
  static constexpr int kN = 8;
  static constexpr bool kNarrow = std::is_same<T, __half>::value;
  using T2 = typename std::conditional<kNarrow, __half2, __nv_bfloat162>::type;
  static __device__ __forceinline__ T2 as2(uint32_t w) { return *reinterpret_cast<T2*>(&w); }
  static __device__ __forceinline__ uint32_t bits(T2 v) { return *reinterpret_cast<uint32_t*>(&v); }
  // the larger of two vectors' elements, NaN ignored
  static __device__ __forceinline__ uint4 vmax(uint4 a, uint4 b) {
    return make_uint4(bits(__hmax2(as2(a.x), as2(b.x))), bits(__hmax2(as2(a.y), as2(b.y))),
                      bits(__hmax2(as2(a.z), as2(b.z))), bits(__hmax2(as2(a.w), as2(b.w))));
  }
  static __device__ __forceinline__ uint4 lowest() {
    const uint32_t w = kNarrow ? 0xfc00fc00u : 0xff80ff80u;  // -inf
    return make_uint4(w, w, w, w);
  }
  static __device__ __forceinline__ float reduce(uint4 a) {
    const T2 m = __hmax2(__hmax2(as2(a.x), as2(a.y)), __hmax2(as2(a.z), as2(a.w)));
    const float2 f = Type16<T>::unpack2(bits(m));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ uint4 keep(uint4 a, int n) {  // the first n elements, 0 < n < 8
    const uint4 l = lowest();
    auto one = [&](uint32_t w, uint32_t low, int left) {
      return left >= 2 ? w : left == 1 ? (w & 0xffffu) | (low & 0xffff0000u) : low;
    };
    return make_uint4(one(a.x, l.x, n), one(a.y, l.y, n - 2), one(a.z, l.z, n - 4), one(a.w, l.w, n - 6));
  }
  static __device__ __forceinline__ float2 two(uint32_t w) {
    if constexpr (kNarrow) return Type16<T>::unpack2(w);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ void unpack(uint4 a, float (&x)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = two(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  // pairs, with -inf raised to a finite value whose exponential is still 0
  // (fp16 -65504, bf16 about -1e38); NaN stays NaN
  static __device__ __forceinline__ void pairs(uint4 a, float2 (&x)[4]) {
    const uint32_t c = kNarrow ? 0xfbfffbffu : 0xfe96fe96u;
    x[0] = two(bits(__hmax2_nan(as2(a.x), as2(c))));
    x[1] = two(bits(__hmax2_nan(as2(a.y), as2(c))));
    x[2] = two(bits(__hmax2_nan(as2(a.z), as2(c))));
    x[3] = two(bits(__hmax2_nan(as2(a.w), as2(c))));
  }
};
template <>
struct Row16<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ uint4 vmax(uint4 a, uint4 b) {
    return make_uint4(one(a.x, b.x), one(a.y, b.y), one(a.z, b.z), one(a.w, b.w));
  }
  static __device__ __forceinline__ uint32_t one(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ uint4 lowest() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
  static __device__ __forceinline__ float reduce(uint4 a) {
    return fmaxf(fmaxf(__uint_as_float(a.x), __uint_as_float(a.y)),
                 fmaxf(__uint_as_float(a.z), __uint_as_float(a.w)));
  }
  static __device__ __forceinline__ uint4 keep(uint4 a, int n) {  // the first n elements, 0 < n < 4
    const uint4 l = lowest();
    return make_uint4(a.x, n > 1 ? a.y : l.y, n > 2 ? a.z : l.z, l.w);
  }
  static __device__ __forceinline__ void unpack(uint4 a, float (&x)[4]) {
    x[0] = __uint_as_float(a.x);
    x[1] = __uint_as_float(a.y);
    x[2] = __uint_as_float(a.z);
    x[3] = __uint_as_float(a.w);
  }
  static __device__ __forceinline__ float raise(uint32_t a) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(__uint_as_float(a)), "f"(-1e38f));
    return d;
  }
  static __device__ __forceinline__ void pairs(uint4 a, float2 (&x)[2]) {
    x[0] = make_float2(raise(a.x), raise(a.y));
    x[1] = make_float2(raise(a.z), raise(a.w));
  }
};

// The alternatives by top_n passes over the row in memory: for rows where more
// logits reach the bound than are kept.  One warp.
template <typename T>
__device__ __noinline__ void top_by_passes(const T* z, int V, int top_n, float m, float log_s, int32_t* ids,
                                           float* lps) {
  using R = Row16<T>;
  constexpr int kN = R::kN;
  const int lane = threadIdx.x & 31, vecs = (V + kN - 1) / kN;
  Cand last{INFINITY, -1};
  for (int k = 0; k < top_n; ++k) {
    Cand best{-INFINITY, 0x7fffffff};
#pragma unroll 4
    for (int v = lane; v < vecs; v += 32) {
      float x[kN];
      R::unpack(*reinterpret_cast<const uint4*>(z + static_cast<long long>(v) * kN), x);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const Cand c{x[i] == x[i] ? x[i] : -INFINITY, v * kN + i};
        if (c.i < V && ahead(last, c) && ahead(c, best)) best = c;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Cand c{__shfl_xor_sync(0xffffffffu, best.v, o), __shfl_xor_sync(0xffffffffu, best.i, o)};
      if (ahead(c, best)) best = c;
    }
    last = best;
    if (lane == 0) {
      ids[k] = best.i;
      lps[k] = (to_f32<T>(z[best.i]) - m) - log_s;
    }
  }
}

// The alternatives from rank `at` on are the lowest ids among the logits equal
// to `value` (-inf: also NaN, which ranks with it).  One warp.
template <typename T>
__device__ void top_equal(const T* z, int V, int top_n, int at, float value, float m, float log_s, int32_t* ids,
                          float* lps) {
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < V && at < top_n; i0 += 32) {
    const float x = i0 + lane < V ? to_f32<T>(z[i0 + lane]) : 0.f;
    const bool take = i0 + lane < V && (value == -INFINITY ? !(x > -INFINITY) : x == value);
    const unsigned who = __ballot_sync(0xffffffffu, take);
    const int k = at + __popc(who & ((1u << lane) - 1));
    if (take && k < top_n) {
      ids[k] = i0 + lane;
      lps[k] = (x - m) - log_s;
    }
    at += __popc(who);
  }
}

// A CTA takes one row after another; each of its 16 warps takes a slice of the
// row through a part of shared memory of its own, whole or, if it is long, in
// chunks.  Of a chunk the warp takes the lanes' maxima, then the sums against
// the largest logit it has seen (two passes over shared memory), and has its
// place filled again by a bulk copy, with the next row's at the end.  So every
// logit is read from memory once, and no warp waits for another to load.
//
// The alternatives: of each row the lanes hand on their maxima.  One more warp
// finds, by bisection, a value that at least top_n of the 512 reach and few more;
// it is no larger than the top_n-th largest logit, and is given out as a
// bound.  The warps look again (in L2) at the few vectors of lanes whose own
// maximum reaches it, for candidates, and hand on their sums; they do so when
// they are through with the next row, so that nobody waits for the bound while
// loads could run.  A last warp joins the sums of a row in a fixed order and
// ranks its candidates.  What crosses between the warps is kept twice, row by
// row in turn: row r is finished before the bound of row r + 2 is given out,
// and nothing of row r + 2 but its maxima is written before that.
//
// Measured at 8192 x 50257 in bf16 with 20 alternatives: 153 us, 5.4 TB/s (three
// passes over memory and L2 took 283).  16 200 warp instructions a row
// keep two thirds of the issue slots busy, and a warp's place lies empty from
// the end of one copy to the end of the sums; two and three smaller places for
// each warp fill that gap but take more instructions, chunk by chunk (203 and
// 229 us).  Without the second look at the candidates it would be 131.  Likely
// tokens that stand together are one warp's to look at again: logits that fall
// by 1e-3 an id take 300 us.  Rows dealt out to the warps in pieces of 512
// bytes took 195 for those, and 169 where nothing falls.  Rows in which fewer
// than top_n lanes hold anything but -inf have a bound of -inf, which all lanes
// reach; they go the way of ties, by one warp over the row once more: 3.3 ms
// with all but 10 logits of a row masked (0.16 ms for 5 alternatives of those).
constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kScoreThreads = kThreads + 64;  // and two warps that see to the rows' ends
constexpr int kKeep = 512;                    // candidates per row
constexpr int kFlood = 96;                    // lanes at the bound that make it a row of ties
constexpr int kRingMany = 100 * 1024;         // two CTAs an SM
constexpr int kRingFew = 200 * 1024;          // one, when there are no more rows than SMs

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

template <typename T>
struct ScoreArgs {
  const T* logits;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  float* lse;
  int32_t* top_ids;
  float* top_logprobs;
  unsigned* err;
  long long ld;
  int M, V, top_n;
  int slice, chunk;  // vectors of a warp, and of one of its slots
};

// Sums against a maximum m (0 in its place when it is -inf): sum = sum
// e^(x - m), dot = sum e^(x - m) (x - m).
struct Sums {
  float m, sum, dot;
};

// The same sums against a larger maximum.
__device__ __forceinline__ void raise(Sums& r, float m) {
  if (r.m == m) return;
  const float down = fmaxf(r.m - m, -1e4f), f = ex2_approx(down * 1.4426950408889634f);  // (0 at -1e4)
  r.dot = fmaf(down, r.sum, r.dot) * f;
  r.sum *= f;
  r.m = m;
}

// Adds this lane's vectors of a chunk to its sums, which are against a maximum
// not below any of them.
template <typename T>
__device__ __forceinline__ void add_chunk(const uint4* chunk, int cnt, Sums& r) {
  using R = Row16<T>;
  constexpr int kN = R::kN;
  const int lane = threadIdx.x & 31;
  constexpr float kL2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  if (fabsf(r.m) < 1e4f) {
    // t = x log2(e) - c in one rounding, c = m log2(e) rounded; what c lost is
    // put right in the sums
    const float c = r.m * kL2e, lost = fmaf(r.m, -kL2e, c);  // t is too small by `lost`
    const float2 neg = make_float2(-c, -c), l2e = make_float2(kL2e, kL2e);
    float2 sum = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int v = lane; v < cnt; v += 32) {
      float2 x[kN / 2];
      R::pairs(chunk[v], x);
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        const float2 t = fma_f32x2(x[i], l2e, neg);
        const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
        sum = add_f32x2(sum, e);
        dot = fma_f32x2(e, t, dot);
      }
    }
    const float f = fmaf(lost, kLn2, 1.f), s = (sum.x + sum.y) * f;  // f = 2^lost
    r.sum += s;
    r.dot = fmaf(fmaf(lost, s, (dot.x + dot.y) * f), kLn2, r.dot);
  } else {  // a maximum far out (or none): `lost` is no small number, differences may overflow
    const float ref = r.m == -INFINITY ? 0.f : r.m;
    for (int v = lane; v < cnt; v += 32) {
      float x[kN];
      R::unpack(chunk[v], x);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float d = x[i] - ref, e = ex2_approx(d * kL2e);
        r.sum += e;
        r.dot = fmaf(e, fmaxf(d, -256.f), r.dot);  // e is 0 there; 0 times -inf would not be
      }
    }
  }
}

// Unsigned keys in the order of the floats (both zeros alike).
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Leaves of the candidates those that reach a value which top_n of them do, and
// not many more (but for ties); returns how many.  Ranking compares all with
// all.  One warp, at most kKeep candidates, at least top_n.
constexpr int kRanked = 64;
__device__ __noinline__ int fewer(Cand* s_cand, int found, int top_n) {
  const int lane = threadIdx.x & 31;
  unsigned low = 0, high = 0xffffffffu;  // low: reached by top_n candidates, high: by fewer
  while (high - low > 1) {
    const unsigned mid = low + (high - low) / 2;
    int n = 0;
    for (int i = 0; i < found; i += 32)
      n += __popc(__ballot_sync(0xffffffffu, i + lane < found && key_of(s_cand[i + lane].v) >= mid));
    if (n >= top_n) {
      low = mid;
      if (n <= kRanked) break;
    } else {
      high = mid;
    }
  }
  int kept = 0;
  for (int i = 0; i < found; i += 32) {
    const Cand c = i + lane < found ? s_cand[i + lane] : Cand{0.f, 0};
    const bool stay = i + lane < found && key_of(c.v) >= low;
    const unsigned who = __ballot_sync(0xffffffffu, stay);
    if (stay) s_cand[kept + __popc(who & ((1u << lane) - 1))] = c;  // (never ahead of what is read)
    kept += __popc(who);
    __syncwarp();
  }
  return kept;
}

// Logits above `bound` anywhere in the row, as candidates; returns their
// number.  One warp.
template <typename T>
__device__ __noinline__ int collect_above(const T* z, int V, float bound, Cand* s_cand, int* s_count, int keep) {
  using R = Row16<T>;
  constexpr int kN = R::kN;
  const int lane = threadIdx.x & 31, vecs = (V + kN - 1) / kN;
  if (lane == 0) *s_count = 0;
  __syncwarp();
#pragma unroll 4
  for (int v = lane; v < vecs; v += 32) {
    float x[kN];
    R::unpack(*reinterpret_cast<const uint4*>(z + static_cast<long long>(v) * kN), x);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (x[i] > bound && v * kN + i < V) {
        const int at = atomicAdd(s_count, 1);
        if (at < keep) s_cand[at] = {x[i], v * kN + i};
      }
  }
  __syncwarp();
  return *s_count;
}

// The outputs of a row from its sums r (against its maximum), and from its
// candidates (s_count of them; at most `keep` are there), which are all logits
// not below `bound`.  One warp.
template <typename T>
__device__ __forceinline__ void put_row(const ScoreArgs<T>& a, int row, const Sums& r, float z_tok, float bound,
                                        Cand* s_cand, int* s_count, int keep) {
  const int lane = threadIdx.x & 31;
  const float m = r.m, log_s = m > -INFINITY ? logf(r.sum) : NAN;
  if (lane == 0) {
    if (a.lse) a.lse[row] = m + log_s;
    if (a.entropy) a.entropy[row] = log_s - r.dot / r.sum;
    if (a.logprob) a.logprob[row] = (z_tok - m) - log_s;
  }
  if (a.top_n == 0) return;
  const T* z = a.logits + row * a.ld;
  int32_t* ids = a.top_ids + static_cast<long long>(row) * a.top_n;
  float* lps = a.top_logprobs + static_cast<long long>(row) * a.top_n;
  int found = *s_count;
  float rest = -INFINITY;  // what the list is filled up with
  if (found > keep) {      // ties at the bound: those above it, then the lowest ids among the ties
    __syncwarp();
    found = collect_above(z, a.V, bound, s_cand, s_count, keep);
    rest = bound;
  }
  if (found > keep) {
    top_by_passes(z, a.V, a.top_n, m, log_s, ids, lps);
  } else {
    if (found > kRanked) found = fewer(s_cand, found, a.top_n);
    for (int k = lane; k < found; k += 32) {
      const Cand c = s_cand[k];
      int at = 0;
#pragma unroll 4
      for (int i = 0; i < found; ++i) at += ahead(s_cand[i], c) ? 1 : 0;
      if (at < a.top_n) {
        ids[at] = c.i;
        lps[at] = (c.v - m) - log_s;
      }
    }
    if (found < a.top_n) top_equal(z, a.V, a.top_n, found, rest, m, log_s, ids, lps);
  }
  __syncwarp();
}

// Short rows: one warp per row, a chunk of four vectors a lane in registers and
// the next on its way.  Each lane keeps sums against a maximum of its own; the bound
// comes from 64 groups' maxima (two a lane) by bisection, and what reaches it
// is looked at again.  A row's end costs the CTA of the kernel below about 3.7
// us: 8192 rows in bf16 take it 110 us at 8000 logits a row (here 68), 122 at
// 14000 (here 93), 143 at 30000 (here 186).  A few rows of 8000 are better off
// with a CTA each (64 rows: 7.9 us, here 19.7).  Bound by issue: 4880 warp
// instructions a row of 8000, 1540 a row of 1000, of which some 1060 for its end.
constexpr int kShortBytes = 40 * 1024;  // of a row, when there are more rows than the other kernel holds
constexpr int kShortAlways = 8 * 1024;  // under which that kernel's groups have no vector each
constexpr int kShortWarps = 8;
constexpr int kShortKeep = 512;
// Adds four vectors to this lane's sums, which are against a reference r.m that
// the largest logit so far passes by less than 1 (-inf: nothing but -inf or NaN
// so far).  A chunk's sums begin at 0, so that behind a large term the small ones
// add up first: a lane's terms pass through kN * 2 + 1 additions of their chunk
// and one of each chunk, V / 1024 (16 bits) or V / 512 (fp32) of them, where one
// running sum would be V / 64 additions long and lose what is below half its last
// place each time.  When the reference moves, what is there shrinks by e at
// least, and the exponentials' errors with it: all those moves together cost less
// than two.
template <typename T>
__device__ __forceinline__ void add_vectors(const uint4 (&x)[4], Sums& r) {
  using R = Row16<T>;
  constexpr int kN = R::kN;
  constexpr float kL2e = 1.4426950408889634f;
  const float m = R::reduce(R::vmax(R::vmax(x[0], x[1]), R::vmax(x[2], x[3])));
  if (m > r.m + 1.f) {
    if (r.m == -INFINITY)
      r.m = m;  // the sums stay
    else
      raise(r, m);
  }
  const float ref = r.m == -INFINITY ? 0.f : r.m;
  float2 sum = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
  if (__any_sync(0xffffffffu, r.m > 1e37f || (r.m < -6e4f && r.m > -INFINITY))) {
    // differences may overflow, or -inf, raised, not be far enough below
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float e[kN];
      R::unpack(x[k], e);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float d = e[i] - ref, p = ex2_approx(d * kL2e);
        float &to = i & 1 ? sum.y : sum.x, &dots = i & 1 ? dot.y : dot.x;
        to += p;
        dots = fmaf(p, fmaxf(d, -256.f), dots);
      }
    }
  } else {
    const float2 neg = make_float2(-ref, -ref), l2e = make_float2(kL2e, kL2e);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 v[kN / 2];
      R::pairs(x[k], v);
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        const float2 d = add_f32x2(v[i], neg), t = mul_f32x2(d, l2e);
        const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
        sum = add_f32x2(sum, e);
        dot = fma_f32x2(e, d, dot);
      }
    }
  }
  r.sum += sum.x + sum.y;
  r.dot += dot.x + dot.y;
}

template <typename T>
__global__ void __launch_bounds__(kShortWarps * 32, 4) score_short(const ScoreArgs<T> a) {
  __shared__ Cand s_cand[kShortWarps][kShortKeep];
  __shared__ int s_count[kShortWarps];
  __shared__ uint8_t s_who[kShortWarps][64];  // a row's groups at the bound
  using R = Row16<T>;
  constexpr int kN = R::kN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vecs = (a.V + kN - 1) / kN, pad = a.V % kN;
  griddep_wait();
  griddep_launch_dependents();
  const int step = gridDim.x * kShortWarps;
  for (int row = blockIdx.x * kShortWarps + warp; row < a.M; row += step) {
    const T* z = a.logits + row * a.ld;
    const uint4* zv = reinterpret_cast<const uint4*>(z);
    const int tok = a.logprob ? a.tokens[row] : 0;
    auto load = [&](int c, uint4 (&x)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int v = c + 32 * k + lane;
        x[k] = v < vecs ? zv[v] : R::lowest();
        if (pad && v == vecs - 1) x[k] = R::keep(x[k], pad);  // what stands behind the vocabulary
      }
    };
    Sums r{-INFINITY, 0.f, 0.f};
    uint4 g0 = R::lowest(), g1 = R::lowest();
    uint4 x[4], y[4];
    load(0, x);
    for (int c = 0; c < vecs; c += 128) {
      if (c + 128 < vecs) load(c + 128, y);
      g0 = R::vmax(g0, R::vmax(x[0], x[2]));
      g1 = R::vmax(g1, R::vmax(x[1], x[3]));
      add_vectors<T>(x, r);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = y[k];
    }
    const bool tok_ok = tok >= 0 && tok < a.V;
    if (!tok_ok && lane == 0) record_error(a.err, kErrRange, kSiteScoreToken);
    const float z_tok = tok_ok ? to_f32<T>(z[tok]) : NAN;
    const float f0 = R::reduce(g0), f1 = R::reduce(g1);  // the groups' maxima
    float m = fmaxf(f0, f1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (r.m > -INFINITY) raise(r, m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      r.sum += __shfl_xor_sync(0xffffffffu, r.sum, o);
      r.dot += __shfl_xor_sync(0xffffffffu, r.dot, o);
    }
    r.m = m;
    float bound = -INFINITY;
    if (a.top_n > 0) {
      // a value that at least top_n groups reach, and few more than that
      const unsigned k0 = key_of(f0), k1 = key_of(f1);
      unsigned low = key_of(-INFINITY), high = key_of(m) + 1;  // low: reached by top_n groups, high: by none
      for (int i = 0; i < 32 && high - low > 1; ++i) {
        const unsigned mid = low + (high - low) / 2;
        const int n = __popc(__ballot_sync(0xffffffffu, k0 >= mid)) + __popc(__ballot_sync(0xffffffffu, k1 >= mid));
        if (n >= a.top_n) {
          low = mid;
          if (n <= a.top_n + 2) break;
        } else {
          high = mid;
        }
      }
      bound = low & 0x80000000u ? __uint_as_float(low & 0x7fffffffu) : __uint_as_float(~low);
      const float least = fmaxf(bound, -3.402823466e38f);  // (-inf is no candidate)
      if (lane == 0) s_count[warp] = 0;
      __syncwarp();
      const unsigned who0 = __ballot_sync(0xffffffffu, f0 >= least), who1 = __ballot_sync(0xffffffffu, f1 >= least);
      const int n0 = __popc(who0), below = (1u << lane) - 1;
      if (who0 >> lane & 1) s_who[warp][__popc(who0 & below)] = static_cast<uint8_t>(lane);
      if (who1 >> lane & 1) s_who[warp][n0 + __popc(who1 & below)] = static_cast<uint8_t>(32 + lane);
      __syncwarp();
      const int each = (vecs + 63) / 64;  // vectors of a group
      for (int t = lane; t < (n0 + __popc(who1)) * each; t += 32) {
        const int f = t / each, v = s_who[warp][f] + 64 * (t - f * each);
        if (v >= vecs) continue;
        const uint4 u = zv[v];
        if (R::reduce(u) < bound && v + 1 < vecs) continue;
        float e[kN];
        R::unpack(u, e);
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (e[i] >= least && v * kN + i < a.V) {
            const int at = atomicAdd(&s_count[warp], 1);
            if (at < kShortKeep) s_cand[warp][at] = {e[i], v * kN + i};
          }
      }
    }
    __syncwarp();
    put_row(a, row, r, z_tok, bound, s_cand[warp], &s_count[warp], kShortKeep);
  }
}

template <typename T>
__global__ void __launch_bounds__(kScoreThreads, 2) score_rows(const ScoreArgs<T> a) {
  extern __shared__ __align__(128) uint8_t s_row[];  // [kWarps][chunk] vectors
  __shared__ Sums s_sums[2][kWarps];
  __shared__ Cand s_cand[2][kKeep];
  __shared__ float s_lane[2][kThreads];  // the lanes' maxima
  __shared__ int s_count[2];
  __shared__ float s_bound[2], s_real[2];  // what the warps compare with, and what it is
  // of even and of odd rows (a warp may be a row ahead of another, never two):
  // maxima there, bound given out, settled, finished
  __shared__ __align__(8) uint64_t s_load[kWarps], s_max[2], s_bnd[2], s_set[2], s_fin[2];
  using R = Row16<T>;
  constexpr int kN = R::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int first = static_cast<int>(blockIdx.x), step = static_cast<int>(gridDim.x);
  const int vecs = (a.V + kN - 1) / kN;
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w) mbar_init(smem_u32(&s_load[w]), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_max[i]), kWarps);
      mbar_init(smem_u32(&s_bnd[i]), 1);
      mbar_init(smem_u32(&s_set[i]), kWarps);
      mbar_init(smem_u32(&s_fin[i]), 1);
    }
    fence_barrier_init();
    s_count[0] = s_count[1] = 0;
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  if (warp < kWarps) {
    // this warp's vectors of a row
    const int v0 = warp * a.slice;
    const int cnt = max(0, min(a.slice, vecs - v0));
    const int pad = (a.V % kN) && cnt > 0 && v0 + cnt == vecs ? a.V % kN : 0;  // elements of the last vector
    const int chunks = (cnt + a.chunk - 1) / a.chunk;
    uint4* chunk = reinterpret_cast<uint4*>(s_row) + warp * a.chunk;
    const uint32_t bar = smem_u32(&s_load[warp]);
    int f_row = first, f_chunk = 0;  // the chunk to fetch next
    auto fetch = [&] {               // lane 0
      if (f_row >= a.M) return;
      const int n = min(a.chunk, cnt - f_chunk * a.chunk);
      mbar_arrive_expect_tx(bar, n * 16);
      bulk_load(smem_u32(chunk), a.logits + f_row * a.ld + (static_cast<long long>(v0) + f_chunk * a.chunk) * kN,
                n * 16, bar);
      if (++f_chunk == chunks) {
        f_chunk = 0;
        f_row += step;
      }
    };
    if (lane == 0 && cnt > 0) fetch();
    int it = 0, parity = 0;
    bool ok = true;
    float mine = -INFINITY;  // this lane's maximum
    Sums r{-INFINITY, 0.f, 0.f};
    auto arrive = [&](uint64_t* bars, int k) {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars[k & 1]));
    };
    auto warp_max = [](float m) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      return m;
    };
    auto hand_on = [&](int k, float m) {  // the lanes' maxima, for the bound
      s_lane[k & 1][tid] = m;
      arrive(s_max, k);
    };
    // Of the row before: candidates among what reaches its bound, and its sums.
    // `k`: the number of that row here.
    auto settle = [&](int row, int k, float mine, const Sums& r) {
      const int buf = k & 1;
      ok = mbar_wait(smem_u32(&s_bnd[buf]), (k >> 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) record_error(a.err, kErrTimeout, kSiteScoreJoin);
        return;
      }
      const float bound = s_bound[buf];
      const float least = fmaxf(bound, -3.402823466e38f);  // (-inf is no candidate)
      unsigned who = __ballot_sync(0xffffffffu, mine >= bound && mine > -INFINITY);
      // the chunks have gone: the vectors of these lanes come from L2, half a
      // warp for each lane
      const uint4* z = reinterpret_cast<const uint4*>(a.logits + row * a.ld) + v0;
      while (who) {
        const int f0 = __ffs(who) - 1;
        who &= who - 1;
        const int f1 = who ? __ffs(who) - 1 : cnt;  // (cnt: none)
        who &= who - 1;
        const int f = lane < 16 ? f0 : f1;
        for (int c = 0; c < cnt; c += a.chunk)
          for (int v = c + f + 32 * (lane & 15); v < min(cnt, c + a.chunk); v += 32 * 16) {
            const uint4 u = z[v];
            if (R::reduce(u) < bound && v + 1 < cnt) continue;
            float x[kN];
            R::unpack(u, x);
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (x[i] >= least && (v + 1 < cnt || !pad || i < pad)) {
                const int at = atomicAdd(&s_count[buf], 1);
                if (at < kKeep) s_cand[buf][at] = {x[i], (v0 + v) * kN + i};
              }
          }
        __syncwarp();
      }
      if (lane == 0) s_sums[buf][warp] = r;
      arrive(s_set, k);
    };
    for (int row = first; row < a.M; row += step, ++it) {
      const float mine_was = mine;
      const Sums r_was = r;
      mine = -INFINITY;
      r = Sums{-INFINITY, 0.f, 0.f};
      for (int c = 0; c < chunks; ++c) {
        ok = mbar_wait(bar, parity);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        parity ^= 1;
        const int n = min(a.chunk, cnt - c * a.chunk);
        if (pad && c + 1 == chunks) {  // what stands behind the vocabulary
          T* last = reinterpret_cast<T*>(chunk + n - 1);
          if (lane >= pad && lane < kN) last[lane] = from_f32<T>(-INFINITY);
          __syncwarp();
        }
        uint4 mx = R::lowest();
#pragma unroll 4
        for (int v = lane; v < n; v += 32) mx = R::vmax(mx, chunk[v]);
        mine = fmaxf(mine, R::reduce(mx));
        if (c + 1 == chunks) hand_on(it, mine);
        const float m = warp_max(mine);
        raise(r, m);
        add_chunk<T>(chunk, n, r);
        __syncwarp();
        if (lane == 0) {
          fence_proxy_async_smem();
          fetch();
        }
      }
      if (!ok) {
        if (lane == 0) record_error(a.err, kErrTimeout, kSiteScoreLoad);
        break;
      }
      if (chunks == 0) hand_on(it, mine);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        r.sum += __shfl_xor_sync(0xffffffffu, r.sum, o);
        r.dot += __shfl_xor_sync(0xffffffffu, r.dot, o);
      }
      if (it > 0) settle(row - step, it - 1, mine_was, r_was);
      if (!ok) break;
    }
    if (ok && it > 0) settle(first + (it - 1) * step, it - 1, mine, r);
    // (given up: the copy in flight must not outlive the CTA)
    if (!ok && lane == 0 && cnt > 0) (void)mbar_wait(bar, parity);
  } else {
    bool ok = true;
    auto arrived = [&](uint64_t* bars, int k) {  // every warp has come to row k
      ok = mbar_wait(smem_u32(&bars[k & 1]), (k >> 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) record_error(a.err, kErrTimeout, kSiteScoreJoin);
      return ok;
    };
    if (warp == kWarps) {
      // ---- bounds
      for (int row = first, it = 0; row < a.M; row += step, ++it) {
        const int buf = it & 1;
        if (!arrived(s_max, it)) break;
        // a value that at least top_n lanes' maxima reach, and few more than that
        float bound = NAN;  // nothing reaches it
        bool flood = false;
        if (a.top_n > 0) {
          unsigned key[kWarps], low = 0xffffffffu, high = 0;
#pragma unroll
          for (int i = 0; i < kWarps; ++i) {
            key[i] = key_of(s_lane[buf][i * 32 + lane]);
            low = min(low, key[i]);
            high = max(high, key[i]);
          }
          low = __reduce_min_sync(0xffffffffu, low);  // all of them reach it
          high = __reduce_max_sync(0xffffffffu, high) + 1;  // none does
          int n = kThreads;
          while (high - low > 1 && n > a.top_n + 2) {
            const unsigned mid = low + (high - low) / 2;
            int c = 0;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) c += key[i] >= mid ? 1 : 0;
            c = __reduce_add_sync(0xffffffffu, c);
            if (c >= a.top_n) {
              low = mid;
              n = c;
            } else {
              high = mid;
            }
          }
          bound = low & 0x80000000u ? __uint_as_float(low & 0x7fffffffu) : __uint_as_float(~low);
          flood = n > kFlood;
        }
        if (it > 1) {  // what row it - 2 left in the buffers has been used
          ok = mbar_wait(smem_u32(&s_fin[buf]), ((it >> 1) - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            if (lane == 0) record_error(a.err, kErrTimeout, kSiteScoreJoin);
            break;
          }
        }
        if (lane == 0) {
          // ties by the hundred: nothing is to be collected, the row's end sees to it
          s_bound[buf] = flood ? NAN : bound;
          s_real[buf] = bound;
          if (flood) s_count[buf] = kKeep + 1;
          mbar_arrive(smem_u32(&s_bnd[buf]));
        }
        __syncwarp();
      }
    } else {
      // ---- ends of rows
      const int n = (a.M - first + step - 1) / step;
      int tok_next = a.logprob ? a.tokens[first] : 0;
      for (int it = 0; it < n; ++it) {
        const int buf = it & 1, row = first + it * step;
        const int tok = tok_next;
        const bool tok_ok = tok >= 0 && tok < a.V;
        if (!tok_ok && lane == 0) record_error(a.err, kErrRange, kSiteScoreToken);
        const float z_tok = tok_ok ? to_f32<T>(a.logits[row * a.ld + tok]) : NAN;
        if (a.logprob && it + 1 < n) tok_next = a.tokens[row + step];
        if (!arrived(s_set, it)) break;
        float m = -INFINITY;
        if (lane < kWarps) m = s_sums[buf][lane].m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float s = 0.f, d = 0.f;
        if (lane < kWarps) {
          Sums x = s_sums[buf][lane];
          if (x.m > -INFINITY) raise(x, m);
          s = x.sum;  // (of a warp with nothing but -inf: 0, or NaN)
          d = x.dot;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          s += __shfl_xor_sync(0xffffffffu, s, o);
          d += __shfl_xor_sync(0xffffffffu, d, o);
        }
        put_row(a, row, Sums{m, s, d}, z_tok, s_real[buf], s_cand[buf], &s_count[buf], kKeep);
        if (lane == 0) s_count[buf] = 0;  // next added to behind the bound of two rows on
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_fin[buf]));
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const void* logits, int64_t ld, int64_t M, int V, const int32_t* tokens, float* logprob,
                     float* entropy, float* lse, int top_n, int32_t* top_ids, float* top_logprobs, cudaStream_t s) {
  constexpr int kN = Row16<T>::kN;
  const int vecs = (V + kN - 1) / kN;
  ScoreArgs<T> a;
  a.logits = static_cast<const T*>(logits);
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.err = device_error_word();
  a.ld = ld;
  a.M = static_cast<int>(M);
  a.V = V;
  a.top_n = top_n;
  const long long row_bytes = 16ll * vecs;
  if (row_bytes < kShortAlways || (row_bytes <= kShortBytes && M > 2 * num_sms())) {
    const int64_t most = 4ll * num_sms(), want = (M + kShortWarps - 1) / kShortWarps;
    return launch_pdl(score_short<T>, static_cast<unsigned>(std::min(want, most)), kShortWarps * 32, 0, s, 0, a);
  }
  const int ring = M > num_sms() ? kRingMany : kRingFew;
  a.slice = (vecs + kWarps - 1) / kWarps;
  // one chunk, or several of much the same size in whole vectors of 32 lanes
  const int most = ring / (kWarps * 16), parts = (a.slice + most / 32 * 32 - 1) / (most / 32 * 32);
  a.chunk = a.slice <= most ? a.slice : ((a.slice + parts - 1) / parts + 31) / 32 * 32;
  const size_t smem = static_cast<size_t>(kWarps) * a.chunk * 16;
  auto kern = score_rows<T>;
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingFew);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(M, 2 * num_sms()));
  return launch_pdl(kern, grid, kScoreThreads, smem, s, 0, a);
}

}  // namespace

cudaError_t launch_token_logprobs(const void* logits, int64_t ld, gpt2_dtype logits_t, int64_t M, int V,
                                  const int32_t* tokens, float* logprob, float* entropy, float* lse, int top_n,
                                  int32_t* top_ids, float* top_logprobs, cudaStream_t s) {
  switch (logits_t) {
    case GPT2_F32:
      return launch_t<float>(logits, ld, M, V, tokens, logprob, entropy, lse, top_n, top_ids, top_logprobs, s);
    case GPT2_F16:
      return launch_t<__half>(logits, ld, M, V, tokens, logprob, entropy, lse, top_n, top_ids, top_logprobs, s);
    default:
      return launch_t<__nv_bfloat16>(logits, ld, M, V, tokens, logprob, entropy, lse, top_n, top_ids, top_logprobs,
                                     s);
  }
}

}  // namespace gpt2
