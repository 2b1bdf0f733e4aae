// Scores from stored logits: log probabilities of given tokens, the entropy
// of each row's distribution and its most likely alternatives.
//
//   m = max z, S = sum e^(z - m), lse = m + log S,
//   log p(v) = (z_v - m) - log S, H = log S - sum e^(z - m) (z - m) / S.
//
// Reading the logits once is all that has to move; the arithmetic (a handful
// of operations and one exponential per logit) is of the same order as the
// memory time.
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

// One CTA per row.  Pass 1: the maximum, and the n-th largest of 128 disjoint
// groups' maxima, a lower bound of the row's n-th largest logit.  Pass 2: the
// sums against the maximum, and every logit at or above the bound as a
// candidate; the candidates are ranked among themselves.  Where they do not
// fit, n passes each find the next alternative.
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
    if (warp == 0 && found < top_n) {
      int at = found;
      for (int i0 = 0; i0 < V && at < top_n; i0 += 32) {
        const float x = i0 + lane < V ? to_f32<T>(z[i0 + lane]) : 0.f;
        const bool take = i0 + lane < V && !(x > -INFINITY);
        const unsigned who = __ballot_sync(0xffffffffu, take);
        const int k = at + __popc(who & ((1u << lane) - 1));
        if (take && k < top_n) {
          ids[k] = i0 + lane;
          lps[k] = (x - m) - log_s;
        }
        at += __popc(who);
      }
    }
    return;
  }
  // a great many logits at or above the bound (ties): one pass per alternative
  Cand last{INFINITY, -1};
  for (int k = 0; k < top_n; ++k) {
    Cand best{-INFINITY, 0x7fffffff};
    for (int v = tid; v < vecs; v += kThreads) {
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
    __syncthreads();
    if (lane == 0) s_cand[warp] = best;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w)
      if (ahead(s_cand[w], best)) best = s_cand[w];
    last = best;
    if (tid == 0) {
      ids[k] = best.i;
      lps[k] = (to_f32<T>(z[best.i]) - m) - log_s;
    }
  }
}

template <typename T>
cudaError_t launch_t(const void* logits, int64_t ld, int64_t M, int V, const int32_t* tokens, float* logprob,
                     float* entropy, float* lse, int top_n, int32_t* top_ids, float* top_logprobs, cudaStream_t s) {
  return launch_pdl(token_logprobs<T>, static_cast<unsigned>(M), kThreads, 0, s, 0, static_cast<const T*>(logits),
                    static_cast<long long>(ld), V, tokens, logprob, entropy, lse, top_n, top_ids, top_logprobs,
                    device_error_word());
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
