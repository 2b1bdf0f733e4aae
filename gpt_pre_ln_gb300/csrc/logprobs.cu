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

constexpr int kThreads = 512;
constexpr int kGroups = kThreads / 4;  // threads whose maxima bound the n-th largest logit from below
constexpr int kCand = 1024;            // candidates kept per row

struct Cand {
  float v;
  int i;
};
// the order of the alternatives: larger value first, lower index on ties
__device__ __forceinline__ bool ahead(const Cand& a, const Cand& b) { return a.v > b.v || (a.v == b.v && a.i < b.i); }

template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
  float x[kN];
};
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* row, int v, int V) {
  Vec<T> r;
  const uint4 u = *reinterpret_cast<const uint4*>(row + static_cast<long long>(v) * Vec<T>::kN);
  if constexpr (sizeof(T) == 4) {
    r.x[0] = __uint_as_float(u.x);
    r.x[1] = __uint_as_float(u.y);
    r.x[2] = __uint_as_float(u.z);
    r.x[3] = __uint_as_float(u.w);
  } else {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Type16<T>::unpack2(w[i]);
      r.x[2 * i] = f.x;
      r.x[2 * i + 1] = f.y;
    }
  }
  if ((v + 1) * Vec<T>::kN > V) {  // the row's padding
#pragma unroll
    for (int i = 0; i < Vec<T>::kN; ++i)
      if (v * Vec<T>::kN + i >= V) r.x[i] = -INFINITY;
  }
  return r;
}

__device__ __forceinline__ float block_sum(float v, float* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) s[warp] = v;
  __syncthreads();
  float r = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) r += s[w];
  __syncthreads();
  return r;
}

// The alternatives by top_n passes over the row in memory: for rows where more
// logits reach the bound than are kept.  WARPS warps together (all of a CTA, or
// one).
template <typename T, int WARPS>
__device__ __noinline__ void top_by_passes(const T* z, int V, int top_n, float m, float log_s, int32_t* ids, float* lps,
                                           Cand* s_best) {
  const int lane = threadIdx.x & 31, warp = WARPS > 1 ? threadIdx.x >> 5 : 0;
  constexpr int kN = Vec<T>::kN;
  const int vecs = (V + kN - 1) / kN;
  Cand last{INFINITY, -1};
  for (int k = 0; k < top_n; ++k) {
    Cand best{-INFINITY, 0x7fffffff};
#pragma unroll 4
    for (int v = warp * 32 + lane; v < vecs; v += WARPS * 32) {
      const Vec<T> x = load_vec(z, v, V);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const Cand c{x.x[i] == x.x[i] ? x.x[i] : -INFINITY, v * kN + i};
        if (c.i < V && ahead(last, c) && ahead(c, best)) best = c;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Cand c{__shfl_xor_sync(0xffffffffu, best.v, o), __shfl_xor_sync(0xffffffffu, best.i, o)};
      if (ahead(c, best)) best = c;
    }
    if constexpr (WARPS > 1) {
      __syncthreads();
      if (lane == 0) s_best[warp] = best;
      __syncthreads();
      for (int w = 0; w < WARPS; ++w)
        if (ahead(s_best[w], best)) best = s_best[w];
    }
    last = best;
    if (warp == 0 && lane == 0) {
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

// One CTA per row.  Pass 1: the maximum, and the n-th largest of 128 disjoint
// groups' maxima, a lower bound of the row's n-th largest logit.  Pass 2: the
// sums against the maximum, and every logit at or above the bound as a
// candidate; the candidates are ranked among themselves.
template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs(const T* __restrict__ logits, long long ld, int V,
                                                           const int32_t* __restrict__ tokens,
                                                           float* __restrict__ logprob, float* __restrict__ entropy,
                                                           float* __restrict__ lse, int top_n,
                                                           int32_t* __restrict__ top_ids,
                                                           float* __restrict__ top_logprobs, unsigned* err) {
  __shared__ float s_group[kGroups];
  __shared__ float s_red[kThreads / 32];
  __shared__ Cand s_cand[kCand];
  __shared__ int s_count;
  __shared__ float s_bound;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x;
  const T* z = logits + row * ld;
  constexpr int kN = Vec<T>::kN;
  const int vecs = (V + kN - 1) / kN;

  float g = -INFINITY;
  for (int v = tid; v < vecs; v += kThreads) {
    const Vec<T> x = load_vec(z, v, V);
#pragma unroll
    for (int i = 0; i < kN; ++i) g = fmaxf(g, x.x[i]);
  }
  g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
  g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
  if ((lane & 3) == 0) s_group[tid >> 2] = g;
  if (tid == 0) s_count = 0;
  __syncthreads();
  float m = -INFINITY;
  for (int i = 0; i < kGroups; i += 32) m = fmaxf(m, s_group[i + lane]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (top_n > 0 && tid < kGroups) {
    const float mine = s_group[tid];
    int rank = 0;
    for (int i = 0; i < kGroups; ++i) {
      const float o = s_group[i];
      rank += (o > mine || (o == mine && i < tid)) ? 1 : 0;
    }
    if (rank == top_n - 1) s_bound = mine;
  }
  __syncthreads();
  const float bound = top_n > 0 ? s_bound : INFINITY;

  float sum = 0.f, dot = 0.f;
  for (int v = tid; v < vecs; v += kThreads) {
    const Vec<T> x = load_vec(z, v, V);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float d = x.x[i] - m;
      const float e = ex2_approx(d * 1.4426950408889634f);
      sum += e;
      dot = fmaf(e, fmaxf(d, -256.f), dot);  // e is 0 there; 0 times -inf would not be
      if (top_n > 0 && x.x[i] >= bound && x.x[i] > -INFINITY) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kCand) s_cand[at] = {x.x[i], v * kN + i};
      }
    }
  }
  sum = block_sum(sum, s_red);
  dot = block_sum(dot, s_red);
  const float log_s = logf(sum);
  if (tid == 0) {
    if (lse) lse[row] = m + log_s;
    if (entropy) entropy[row] = log_s - dot / sum;
    if (logprob) {
      const int t = tokens[row];
      if (t >= 0 && t < V) {
        logprob[row] = (to_f32<T>(z[t]) - m) - log_s;
      } else {
        record_error(err, kErrRange, kSiteScoreToken);
        logprob[row] = NAN;
      }
    }
  }
  if (top_n == 0) return;
  const int found = s_count;  // (behind the barriers of block_sum)
  int32_t* ids = top_ids + row * top_n;
  float* lps = top_logprobs + row * top_n;
  if (found <= kCand) {
    for (int k = tid; k < found; k += kThreads) {
      const Cand c = s_cand[k];
      int rank = 0;
      for (int i = 0; i < found; ++i) rank += ahead(s_cand[i], c) ? 1 : 0;
      if (rank < top_n) {
        ids[rank] = c.i;
        lps[rank] = (c.v - m) - log_s;
      }
    }
    // fewer than n: the bound was -inf, every other logit is -inf (or NaN,
    // which ranks with it); the lowest indices among those follow
    if (warp == 0 && found < top_n) top_equal(z, V, top_n, found, -INFINITY, m, log_s, ids, lps);
    return;
  }
  // a great many logits at or above the bound: ties
  top_by_passes<T, kThreads / 32>(z, V, top_n, m, log_s, ids, lps, s_cand);
}

// ------------------------------------------------------- rows kept on chip
// The kernel for rows that fit the shared memory of a cluster: each row is
// read from memory once.  A cluster of C CTAs (1, 2, 4 or 8) holds one row at
// a time, each CTA a part of it and each of its 16 warps a slice of that,
// fetched by the warp's own bulk copy.  Rows are taken one after another.  Per
// row a warp (1) takes the maxima of its slice's lanes and hands on those of 4
// groups of 8 lanes (fewer with several CTAs), (2) sums against its own
// maximum and fetches its slice of the next row, (3) looks again (in L2) at the
// few vectors of lanes whose maximum reaches the bound, for candidates, and
// hands on its sums.  The bound, the top_n-th largest of 64 groups' maxima and
// so no larger than the top_n-th largest logit, comes from one more warp (in
// the cluster's first CTA); (3) waits until the warp has done (1) and (2) of
// the next row, so that nobody waits for the bound while loads could run.  A
// last warp joins the sums of a row in a fixed order and ranks its candidates,
// beside the other warps' work.  What crosses between them is kept twice, row
// by row in turn: row r is finished before the bound of row r + 2 is given
// out, and nothing of row r + 2 but its maxima is written before that.
//
// Measured at 8192 x 50257 in bf16 with 20 alternatives: @@LP@@
constexpr int kWarps = kThreads / 32;
constexpr int kScoreThreads = kThreads + 64;   // and two warps that see to the rows' ends
constexpr int kKeep = 512;                     // candidates per row
constexpr int kPartBytes = 100 * 1024;         // two CTAs of this size share an SM
constexpr int kPartBytesMax = 208 * 1024;      // one does
constexpr int kMaxCluster = 8;
constexpr int kFlood = 16;  // lanes of a warp at the bound that make it a row of ties

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

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ int add_cluster(uint32_t addr, int v) {
  int old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.s32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}
// A bounded wait for a barrier that CTAs of the cluster share.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
    for (int i = 0; i < 32; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}\n"
          : "=r"(ok)
          : "r"(bar), "r"(parity)
          : "memory");
      if (ok) return true;
    }
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}
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
  int part, slice;  // vectors per CTA and per warp
};

// A warp's sums over its slice against its own maximum m (or 0 when there is
// none): sum = sum e^(x - m), dot = sum e^(x - m) (x - m).
struct Sums {
  float m, sum, dot;
};

template <typename T>
__device__ __forceinline__ Sums slice_sums(const uint4* slice, int cnt, float m) {
  using R = Row16<T>;
  constexpr int kN = R::kN;
  const int lane = threadIdx.x & 31;
  constexpr float kL2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  Sums r{m, 0.f, 0.f};
  if (fabsf(m) < 1e4f) {
    // t = x log2(e) - c in one rounding, c = m log2(e) rounded; what c lost is
    // put right in the sums
    const float c = m * kL2e, lost = fmaf(m, -kL2e, c);  // t is too small by `lost`
    const float2 neg = make_float2(-c, -c), l2e = make_float2(kL2e, kL2e);
    float2 sum = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int v = lane; v < cnt; v += 32) {
      float2 x[kN / 2];
      R::pairs(slice[v], x);
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        const float2 t = fma_f32x2(x[i], l2e, neg);
        const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
        sum = add_f32x2(sum, e);
        dot = fma_f32x2(e, t, dot);
      }
    }
    const float f = fmaf(lost, kLn2, 1.f);  // 2^lost
    r.sum = (sum.x + sum.y) * f;
    r.dot = fmaf(lost, r.sum, (dot.x + dot.y) * f) * kLn2;
  } else {  // a maximum far out (or none): `lost` is no small number, differences may overflow
    const float ref = m == -INFINITY ? 0.f : m;
    const T* x = reinterpret_cast<const T*>(slice);
    for (int v = lane; v < cnt * kN; v += 32) {
      const float d = to_f32<T>(x[v]) - ref;
      const float e = ex2_approx(d * kL2e);
      r.sum += e;
      r.dot = fmaf(e, fmaxf(d, -256.f), r.dot);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    r.sum += __shfl_xor_sync(0xffffffffu, r.sum, o);
    r.dot += __shfl_xor_sync(0xffffffffu, r.dot, o);
  }
  return r;
}

// Logits above `bound` anywhere in the row, as candidates; returns their
// number.  One warp.
template <typename T>
__device__ __noinline__ int collect_above(const T* z, int V, float bound, Cand* s_cand, int* s_count) {
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
        if (at < kKeep) s_cand[at] = {x[i], v * kN + i};
      }
  }
  __syncwarp();
  return *s_count;
}

template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kScoreThreads, 2) score_rows(const ScoreArgs<T> a) {
  extern __shared__ __align__(128) uint8_t s_row[];  // [kWarps][slice] vectors
  __shared__ Sums s_sums[2][kMaxCluster * kWarps];
  __shared__ Cand s_cand[2][kKeep];
  __shared__ float s_raw[2][kMaxCluster * kWarps];  // groups' maxima
  __shared__ __align__(16) float s_group[64];
  __shared__ int s_count[2];
  __shared__ float s_bound[2];
  // of even and of odd rows (a warp may be a row ahead of another, never two):
  // maxima there, bound given out, settled, finished
  __shared__ __align__(8) uint64_t s_load[kWarps], s_max[2], s_bnd[2], s_set[2], s_fin[2];
  using R = Row16<T>;
  constexpr int kN = R::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
  const int C = CLUSTER ? static_cast<int>(cluster_nctarank()) : 1;
  const int first = static_cast<int>(blockIdx.x) / C, step = static_cast<int>(gridDim.x) / C;
  const int vecs = (a.V + kN - 1) / kN;
  const int per_warp = C >= 4 ? 1 : 4 / C;  // groups of a warp: 64 in all (128 with eight CTAs)
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w) mbar_init(smem_u32(&s_load[w]), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_max[i]), C * kWarps);
      mbar_init(smem_u32(&s_bnd[i]), 1);
      mbar_init(smem_u32(&s_set[i]), C * kWarps);
      mbar_init(smem_u32(&s_fin[i]), 1);
    }
    fence_barrier_init();
    s_count[0] = s_count[1] = 0;
  }
  if (CLUSTER)
    cluster_sync();
  else
    __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  if (warp < kWarps) {
    // this warp's vectors of a row
    const int v0 = rank * a.part + warp * a.slice;
    const int cnt = max(0, min(min(a.slice, a.part - warp * a.slice), vecs - v0));
    const int pad = (a.V % kN) && cnt > 0 && v0 + cnt == vecs ? a.V % kN : 0;  // elements of the last vector
    uint4* slice = reinterpret_cast<uint4*>(s_row) + warp * a.slice;
    const uint32_t bar = smem_u32(&s_load[warp]);
    auto fetch = [&](int row) {
      mbar_arrive_expect_tx(bar, cnt * 16);
      bulk_load(smem_u32(slice), a.logits + row * a.ld + static_cast<long long>(v0) * kN, cnt * 16, bar);
    };
    if (lane == 0 && cnt > 0 && first < a.M) fetch(first);
    int it = 0;
    bool ok = true;
    float mine = -INFINITY;
    Sums r{-INFINITY, 0.f, 0.f};
    auto arrive = [&](uint64_t* bars, int k) {
      __syncwarp();
      if (lane == 0) {
        const uint32_t b = smem_u32(&bars[k & 1]);
        if (CLUSTER)
          mbar_arrive_cluster(mapa_shared(b, 0));
        else
          mbar_arrive(b);
      }
    };
    // (3) of the row before: candidates among what reaches its bound, and its
    // sums.  `k`: the number of that row here.
    auto settle = [&](int row, int k, float mine, const Sums& r) {
      const int buf = k & 1;
      const uint32_t bnd = smem_u32(&s_bnd[buf]);
      ok = CLUSTER ? mbar_wait_cluster(bnd, (k >> 1) & 1) : mbar_wait(bnd, (k >> 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) record_error(a.err, kErrTimeout, kSiteScoreJoin);
        return;
      }
      const float bound = s_bound[buf];
      unsigned who = __ballot_sync(0xffffffffu, mine >= bound && mine > -INFINITY);
      if (who) {
        // the slice has gone: these few vectors come from L2
        const uint4* z = reinterpret_cast<const uint4*>(a.logits + row * a.ld) + v0;
        const uint32_t count = CLUSTER ? mapa_shared(smem_u32(&s_count[buf]), 0) : 0;
        if (__popc(who) > kFlood) {
          if (lane == 0) {
            if (CLUSTER)
              add_cluster(count, kKeep + 1);
            else
              atomicAdd(&s_count[buf], kKeep + 1);
          }
          who = 0;
        }
        while (who) {
          const int f = __ffs(who) - 1;
          who &= who - 1;
          for (int v = f + 32 * lane; v < cnt; v += 32 * 32) {
            const uint4 u = z[v];
            if (v + 1 < cnt && R::reduce(u) < bound) continue;
            float x[kN];
            R::unpack(u, x);
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (x[i] >= bound && x[i] > -INFINITY && (v0 + v) * kN + i < a.V) {
                const int id = (v0 + v) * kN + i;
                if (CLUSTER) {
                  const int at = add_cluster(count, 1);
                  if (at < kKeep) {
                    const uint32_t to = mapa_shared(smem_u32(&s_cand[buf][at]), 0);
                    st_cluster(to, x[i]);
                    st_cluster(to + 4, id);
                  }
                } else {
                  const int at = atomicAdd(&s_count[buf], 1);
                  if (at < kKeep) s_cand[buf][at] = {x[i], id};
                }
              }
          }
          __syncwarp();
        }
      }
      if (lane == 0) {
        if (CLUSTER) {
          const uint32_t to = mapa_shared(smem_u32(&s_sums[buf][rank * kWarps + warp]), 0);
          st_cluster(to, r.m);
          st_cluster(to + 4, r.sum);
          st_cluster(to + 8, r.dot);
        } else {
          s_sums[buf][warp] = r;
        }
      }
      arrive(s_set, k);
    };
    for (int row = first; row < a.M; row += step, ++it) {
      // ---- (1) maxima
      uint4 mx = R::lowest();
      if (cnt > 0) {
        if (!mbar_wait(bar, it & 1)) {
          if (lane == 0) record_error(a.err, kErrTimeout, kSiteScoreLoad);
          (void)mbar_wait(bar, it & 1);  // the copy must not outlive the CTA
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (pad) {  // what stands behind the vocabulary
          T* last = reinterpret_cast<T*>(slice + cnt - 1);
          if (lane >= pad && lane < kN) last[lane] = from_f32<T>(-INFINITY);
          __syncwarp();
        }
#pragma unroll 4
        for (int v = lane; v < cnt; v += 32) mx = R::vmax(mx, slice[v]);
      }
      const float mine_was = mine;
      const Sums r_was = r;
      mine = R::reduce(mx);
      float m = mine;
#pragma unroll
      for (int o = 1; o <= 32; o <<= 1) {
        if (o * per_warp == 32 && lane % o == 0) {  // m: the maximum of the o lanes from this one on
          float* to = &s_raw[it & 1][(rank * kWarps + warp) * per_warp + lane / o];
          if (CLUSTER)
            st_cluster(mapa_shared(smem_u32(to), 0), m);
          else
            *to = m;
        }
        if (o < 32) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
      arrive(s_max, it);
      // ---- (2) sums, and the next row's slice (the shuffles of the sums are
      // behind every lane's reads of this one)
      r = slice_sums<T>(slice, cnt, m);
      if (lane == 0 && cnt > 0 && row + step < a.M) {
        fence_proxy_async_smem();
        fetch(row + step);
      }
      if (it > 0) settle(row - step, it - 1, mine_was, r_was);
      if (!ok) {
        if (lane == 0 && cnt > 0 && row + step < a.M) (void)mbar_wait(bar, (it + 1) & 1);  // the copy in flight
        break;
      }
    }
    if (ok && it > 0) settle(first + (it - 1) * step, it - 1, mine, r);
  } else if (rank == 0) {
    bool ok = true;
    auto arrived = [&](uint64_t* bars, int k) {  // every warp has come to row k
      const uint32_t b = smem_u32(&bars[k & 1]);
      ok = CLUSTER ? mbar_wait_cluster(b, (k >> 1) & 1) : mbar_wait(b, (k >> 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) record_error(a.err, kErrTimeout, kSiteScoreJoin);
      return ok;
    };
    if (warp == kWarps) {
      // ---- bounds
      const int raw = C * kWarps * per_warp;
      for (int row = first, it = 0; row < a.M; row += step, ++it) {
        const int buf = it & 1;
        if (!arrived(s_max, it)) break;
        float bound = NAN;  // nothing reaches it
        if (a.top_n > 0) {
          float x0 = s_raw[buf][lane], x1 = s_raw[buf][lane + 32];
          if (raw > 64) {
            x0 = fmaxf(x0, s_raw[buf][lane + 64]);
            x1 = fmaxf(x1, s_raw[buf][lane + 96]);
          }
          s_group[lane] = x0;
          s_group[lane + 32] = x1;
          __syncwarp();
          int r0 = 0, r1 = 0;
#pragma unroll 4
          for (int i = 0; i < 64; i += 4) {
            const float4 o = *reinterpret_cast<const float4*>(&s_group[i]);
            const float q[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              r0 += (q[e] > x0 || (q[e] == x0 && i + e < lane)) ? 1 : 0;
              r1 += (q[e] > x1 || (q[e] == x1 && i + e < lane + 32)) ? 1 : 0;
            }
          }
          const unsigned b0 = __ballot_sync(0xffffffffu, r0 == a.top_n - 1);
          const unsigned b1 = __ballot_sync(0xffffffffu, r1 == a.top_n - 1);
          bound = b0 ? __shfl_sync(0xffffffffu, x0, __ffs(b0) - 1) : __shfl_sync(0xffffffffu, x1, __ffs(b1) - 1);
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
          if (CLUSTER) {
            for (int c = 0; c < C; ++c) {
              st_cluster(mapa_shared(smem_u32(&s_bound[buf]), c), bound);
              mbar_arrive_cluster(mapa_shared(smem_u32(&s_bnd[buf]), c));
            }
          } else {
            s_bound[buf] = bound;
            mbar_arrive(smem_u32(&s_bnd[buf]));
          }
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
        for (int i = lane; i < C * kWarps; i += 32) m = fmaxf(m, s_sums[buf][i].m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float s = 0.f, d = 0.f;
        for (int i = lane; i < C * kWarps; i += 32) {
          const Sums x = s_sums[buf][i];
          if (x.m == -INFINITY) {
            s += x.sum;  // 0, or NaN
            continue;
          }
          const float down = fmaxf(x.m - m, -1e4f);  // (its factor is 0 there)
          const float c = ex2_approx(down * 1.4426950408889634f);
          s = fmaf(c, x.sum, s);
          d = fmaf(c, fmaf(down, x.sum, x.dot), d);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          s += __shfl_xor_sync(0xffffffffu, s, o);
          d += __shfl_xor_sync(0xffffffffu, d, o);
        }
        const float log_s = m > -INFINITY ? logf(s) : NAN;
        if (lane == 0) {
          if (a.lse) a.lse[row] = m + log_s;
          if (a.entropy) a.entropy[row] = log_s - d / s;
          if (a.logprob) a.logprob[row] = (z_tok - m) - log_s;
        }
        if (a.top_n > 0) {
          const T* z = a.logits + row * a.ld;
          int32_t* ids = a.top_ids + static_cast<long long>(row) * a.top_n;
          float* lps = a.top_logprobs + static_cast<long long>(row) * a.top_n;
          int found = s_count[buf];
          float rest = -INFINITY;  // what the list is filled up with
          if (found > kKeep) {     // ties at the bound: those above it, then the lowest ids among the ties
            found = collect_above(z, a.V, s_bound[buf], s_cand[buf], &s_count[buf]);
            rest = s_bound[buf];
          }
          if (found > kKeep) {
            top_by_passes<T, 1>(z, a.V, a.top_n, m, log_s, ids, lps, nullptr);
          } else {
            for (int k = lane; k < found; k += 32) {
              const Cand c = s_cand[buf][k];
              int at = 0;
#pragma unroll 4
              for (int i = 0; i < found; ++i) at += ahead(s_cand[buf][i], c) ? 1 : 0;
              if (at < a.top_n) {
                ids[at] = c.i;
                lps[at] = (c.v - m) - log_s;
              }
            }
            if (found < a.top_n) top_equal(z, a.V, a.top_n, found, rest, m, log_s, ids, lps);
          }
          __syncwarp();
          if (lane == 0) s_count[buf] = 0;  // next added to behind the bound of two rows on
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_fin[buf]));
      }
    }
  }
  __syncwarp();
  if (CLUSTER) cluster_sync();  // no CTA leaves while another may still write to it
}

// CTAs per row: the fewest (1, 2, 4, 8) whose parts let two CTAs share an SM,
// and with few rows as many as the SMs hold at two each.  0: the row does not
// fit a cluster.
inline int cluster_for(long long row_bytes, int64_t M) {
  int c = 1;
  while (c < kMaxCluster && row_bytes > static_cast<long long>(c) * kPartBytes) c *= 2;
  if (row_bytes > static_cast<long long>(c) * kPartBytesMax) return 0;
  while (c < kMaxCluster && M * c <= num_sms() && row_bytes > c * 16 * 1024) c *= 2;
  return c;
}

template <typename T>
cudaError_t launch_t(const void* logits, int64_t ld, int64_t M, int V, const int32_t* tokens, float* logprob,
                     float* entropy, float* lse, int top_n, int32_t* top_ids, float* top_logprobs, cudaStream_t s) {
  constexpr int kN = Row16<T>::kN;
  const int vecs = (V + kN - 1) / kN;
  const int C = cluster_for(16ll * vecs, M);
  if (C == 0)
    return launch_pdl(token_logprobs<T>, static_cast<unsigned>(M), kThreads, 0, s, 0, static_cast<const T*>(logits),
                      static_cast<long long>(ld), V, tokens, logprob, entropy, lse, top_n, top_ids, top_logprobs,
                      device_error_word());
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
  a.part = (vecs + C - 1) / C;
  a.slice = (a.part + kWarps - 1) / kWarps;
  const size_t smem = static_cast<size_t>(kWarps) * a.slice * 16;
  auto kern = C > 1 ? score_rows<T, true> : score_rows<T, false>;
  static int configured[2][64] = {{0}};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[C > 1][dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPartBytesMax + 256);
    if (e != cudaSuccess) return e;
    configured[C > 1][dev] = 1;
  }
  const long long fit = std::max(1, 2 * num_sms() / C);
  const unsigned grid = static_cast<unsigned>(std::min<long long>(M, fit) * C);
  return launch_pdl(kern, grid, kScoreThreads, smem, s, C > 1 ? C : 0, a);
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
