// Tokens drawn from stored logits with given random numbers, under a
// temperature, top-k, top-p and min-p.
//
//   w_v = e^((z_v - max z) / temperature)
//
// In the order of falling z (lowest id first on ties) a row keeps the first
// tokens: the top-k first, of those the ones before which less than top_p of
// their weight stands, and those with w >= min_p; all three are a prefix of the
// same order.  The token is where the running sum of the kept weights, in the
// order of the ids, passes uniform times their sum.
//
// An id is right or wrong: a sum in fp32 is off by 1e-7 of itself at best, which is
// more than many a token's share.  So every sum is kept with a bound of its
// error; where a decision lies within it, the row is done once more with weights
// and sums of two floats each (2^-36 of the row's weight at worst, 2^-42 as a
// rule).
//
// One CTA per row, which it reads once into shared memory (rows that do not fit
// are read from global memory, where they stay in L2) and goes over there: the
// maximum; with top-k or top-p a histogram and the elements around the border,
// which are ranked; the sums of the warps' parts of the row; and the part that
// the random number falls into.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace gpt2 {

namespace {

constexpr int kBins = 2048;
constexpr int kList = 512;  // elements that are ranked at a time

// ------------------------------------------------------------ two-float sums
// a value as hi + lo, lo at most half a step of hi
struct Two {
  float hi, lo;
};
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = a + b;
  const float t = s - a;
  e = (a - (s - t)) + (b - t);
}
__device__ __forceinline__ Two norm(float a, float b) {  // |a| >= |b|
  const float s = a + b;
  return {s, b - (s - a)};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  float s, e;
  two_sum(a.hi, b.hi, s, e);
  return norm(s, e + (a.lo + b.lo));
}
__device__ __forceinline__ double value(Two a) { return static_cast<double>(a.hi) + a.lo; }
__device__ __forceinline__ Two shfl_xor(Two a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Two shfl_up(Two a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Two warp_add(Two a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = add(a, shfl_xor(a, o));
  return a;
}

// 2^(k / 64), k = -32 .. 32, as hi + lo
__device__ const float2 kExp2[65] = {
    {0.7071067690849304f, 1.2101617485882343e-08f}, {0.7148066759109497f, -6.714964584375593e-09f}, {0.7225903868675232f, 1.662099968768871e-08f},
    {0.7304589152336121f, -1.814328776106322e-08f}, {0.7384130954742432f, -2.250449426810519e-08f}, {0.7464538812637329f, -1.7118100714696993e-08f},
    {0.7545822262763977f, -1.2479686617439256e-08f}, {0.762799084186554f, -8.814284413460882e-09f}, {0.7711054086685181f, 4.035452416673024e-09f},
    {0.7795022130012512f, -1.2882332534047691e-08f}, {0.7879904508590698f, -2.830512713103417e-08f}, {0.7965710759162903f, -2.451568392736192e-10f},
    {0.8052451610565186f, 4.918108587048664e-09f}, {0.8140137195587158f, -8.630041570256708e-09f}, {0.8228777647018433f, -2.5624860455764065e-08f},
    {0.8318383097648621f, -1.9601493761456368e-08f}, {0.8408964276313782f, -1.2377663338725142e-08f}, {0.8500531911849976f, -1.4325736152898116e-08f},
    {0.8593096733093262f, -2.4248087981959543e-08f}, {0.86866694688797f, -2.9251117084072575e-08f}, {0.8781260848045349f, -4.617885185353998e-09f},
    {0.8876882195472717f, 2.6715989420722508e-08f}, {0.8973545432090759f, -5.707522454656555e-09f}, {0.9071260690689087f, 1.8681291180655535e-08f},
    {0.9170040488243103f, -5.619638976384067e-09f}, {0.9269895553588867f, 7.182805905614487e-09f}, {0.9370838403701782f, -2.331502813035513e-08f},
    {0.9472879767417908f, 1.4051692254213322e-08f}, {0.9576032757759094f, 4.922664054163306e-09f}, {0.9680308699607849f, 2.6785361484371606e-08f},
    {0.9785720705986023f, -8.510902205216553e-09f}, {0.9892280101776123f, 3.0163631592472484e-09f}, {1.0f, 0.0f},
    {1.0108892917633057f, -5.7116054108519165e-09f}, {1.0218971967697144f, -4.811559861650494e-08f}, {1.0330249071121216f, -2.809089316713198e-08f},
    {1.0442737340927124f, 4.8334701574503924e-08f}, {1.055645227432251f, -4.9071694263602694e-08f}, {1.0671404600143433f, -5.9337519786595294e-08f},
    {1.0787607431411743f, 5.4615945543901034e-08f}, {1.0905077457427979f, -1.3077539939843064e-08f}, {1.1023825407028198f, 4.260501995645427e-08f},
    {1.114386796951294f, -5.435540018083884e-08f}, {1.1265215873718262f, 3.12364143439936e-08f}, {1.1387885808944702f, 5.386222312608879e-08f},
    {1.1511892080307007f, 2.1922282655850722e-08f}, {1.1637248992919922f, -4.051441493402308e-08f}, {1.1763969659805298f, 2.566975076945255e-08f},
    {1.1892070770263672f, 3.797635272917432e-08f}, {1.2021567821502686f, -5.069756525699631e-08f}, {1.215247392654419f, -3.267394887984665e-08f},
    {1.228480577468872f, -4.136200359994291e-08f}, {1.2418577671051025f, 4.496838101886169e-08f}, {1.2553807497024536f, 7.3222374830095305e-09f},
    {1.2690509557724f, 1.419333317542737e-09f}, {1.2828700542449951f, -3.816621685359678e-08f}, {1.2968395948410034f, -4.018999533172973e-08f},
    {1.3109612464904785f, -3.496571565619888e-08f}, {1.3252366781234741f, -3.496373324196611e-08f}, {1.339667558670044f, -3.4616739696957666e-08f},
    {1.3542555570602417f, -1.0123349269974824e-08f}, {1.3690024614334106f, -3.845881835218279e-08f}, {1.3839099407196045f, -5.875577357983275e-08f},
    {1.398979663848877f, 8.689434061182055e-09f}, {1.4142135381698608f, 2.4203234971764687e-08f}
};

// The row's scale: t = (z - max) log2(e) / temperature = (z/2 - max/2) c (half
// of each, so that the difference of any two is a number).
struct Scale {
  float half_max, c_hi, c_lo;
};

// w = 2^t to fp32 accuracy: t is off by three roundings, the exponential by 2^-22.
__device__ __forceinline__ float weight1(const Scale& s, float z, float& t) {
  t = (0.5f * z - s.half_max) * s.c_hi;
  return ex2_approx(t);
}
constexpr float kErrExp = 4.5e-7f;   // 2^-22, and three roundings of a sum of eight
constexpr float kErrArg = 1.25e-7f;  // per unit of |t|: 3 * 2^-24 * ln 2

// The same to about 2^-45 of itself: t as two floats, 2^t = 2^n 2^(k/64) e^x with
// the integer n, the nearest k and |x| <= ln 2 / 128, whose series ends with x^5.
// Weights below 2^-100 count as 0.
__device__ __forceinline__ Two weight2(const Scale& s, const float2* table, float z) {
  const float a = 0.5f * z;
  float d, d_lo;
  two_sum(a, -s.half_max, d, d_lo);
  const float t = d * s.c_hi;
  if (!(t > -100.f)) return {0.f, 0.f};
  const float t_lo = fmaf(d, s.c_hi, -t) + fmaf(d, s.c_lo, d_lo * s.c_hi);
  const float n = rintf(t), f = t - n, k = rintf(64.f * f), g = fmaf(k, -0.015625f, f);
  constexpr float kLn2Hi = 0.6931471824645996f, kLn2Lo = -1.9046542121259336e-09f;  // ln 2
  const float x = g * kLn2Hi;
  const float x_lo = fmaf(g, kLn2Hi, -x) + fmaf(g, kLn2Lo, t_lo * kLn2Hi);
  const float h = 0.5f * x, q = h * x;
  const float q_lo = fmaf(h, x, -q) + x * x_lo;
  const float p = x * x * x * fmaf(x, fmaf(x, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f);
  const Two y = norm(x, q);  // e^x - 1
  const float y_lo = y.lo + (x_lo + q_lo + p);
  const float2 b = table[static_cast<int>(k) + 32];
  const float m = b.x * y.hi;
  const float m_lo = fmaf(b.x, y.hi, -m) + fmaf(b.x, y_lo, fmaf(b.y, y.hi, b.y));
  const Two w = norm(b.x, m);
  const Two r = norm(w.hi, w.lo + m_lo);
  const float scale = __int_as_float((static_cast<int>(n) + 127) << 23);
  return {r.hi * scale, r.lo * scale};
}

// Elements in order: larger z first, lowest id first on ties, as one number
// that falls.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);  // -0 counts as 0
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float z_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ unsigned long long place_of(uint32_t key, int id) {
  return (static_cast<unsigned long long>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}
// 16 bytes of a row
template <typename T>
struct Vec {
  static constexpr int kN = 16 / static_cast<int>(sizeof(T));
  static __device__ __forceinline__ void unpack(const uint4& u, float (&z)[kN]) {
    if constexpr (sizeof(T) == 4) {
      z[0] = __uint_as_float(u.x), z[1] = __uint_as_float(u.y), z[2] = __uint_as_float(u.z),
      z[3] = __uint_as_float(u.w);
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = Type16<T>::unpack2(w[i]);
        z[2 * i] = f.x;
        z[2 * i + 1] = f.y;
      }
    }
  }
};

struct SampleArgs {
  const void* logits;
  long long ld;
  int V;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniform;
  int32_t* tokens;
  float* logprob;
  unsigned* err;
};

// What a CTA knows of its row, and its shared memory.
template <typename T>
struct Row {
  const uint4* v;  // the row, in shared or global memory
  int V, vecs, per_warp;  // vectors of the row, and of one warp's part
  Scale scale;
  uint32_t* hist;              // [kBins]
  unsigned long long* list;    // [kList]
  unsigned long long* sorted;  // [kList], in the place of hist
};
struct Shared {
  Two part[32];
  float aux[32];
  int num[32];
  uint32_t lo, hi;
  int count, first, last;
  float before;
  unsigned long long cut;
  Two kept, above;
  float loose;
  int found;
  float2 table[65];
};

// The elements of this warp's part of the row, a lane's vector at a time.
template <typename T, typename F>
__device__ __forceinline__ void each(const Row<T>& r, int from, int to, F&& f) {
  constexpr int kN = Vec<T>::kN;
  const int lane = threadIdx.x & 31;
  for (int v = from + lane; v < to; v += 32) {
    float z[kN];
    Vec<T>::unpack(r.v[v], z);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (v * kN + i >= r.V) z[i] = -INFINITY;  // behind the row: nothing
    f(z, v * kN);
  }
}
template <typename T, typename F>
__device__ __forceinline__ void each_of_part(const Row<T>& r, F&& f) {
  const int from = (threadIdx.x >> 5) * r.per_warp;
  each(r, min(from, r.vecs), min(from + r.per_warp, r.vecs), f);
}

// Sum of this lane's weights over elements at or above `cut`, in the order of
// the ids; err adds the bound of its error (fp32 weights only).
template <bool TWO, typename T>
struct Weights {
  const Row<T>& r;
  const float2* table;
  Two sum{0.f, 0.f};
  float wt = 0.f;  // sum of w |t|
  __device__ __forceinline__ Weights(const Row<T>& row, const float2* tab) : r(row), table(tab) {}
  __device__ __forceinline__ void add_vec(const float (&z)[Vec<T>::kN], int id, unsigned long long cut) {
    constexpr int kN = Vec<T>::kN;
    const uint32_t key_cut = static_cast<uint32_t>(cut >> 32);
    if constexpr (TWO) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t key = key_of(z[i]);
        if (key > key_cut || (key == key_cut && place_of(key, id + i) >= cut)) sum = add(sum, weight2(r.scale, table, z[i]));
      }
    } else {
      float w[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t key = key_of(z[i]);
        float t;
        w[i] = weight1(r.scale, z[i], t);
        if (!(key > key_cut || (key == key_cut && place_of(key, id + i) >= cut))) w[i] = 0.f;
        if (w[i] > 0.f) wt = fmaf(w[i], -t, wt);
      }
#pragma unroll
      for (int o = 1; o < kN; o <<= 1)
#pragma unroll
        for (int i = 0; i < kN; i += 2 * o) w[i] += w[i + o];
      float s, e;
      two_sum(sum.hi, w[0], s, e);
      sum = {s, sum.lo + e};
    }
  }
  __device__ __forceinline__ float error() const { return TWO ? 0.f : fmaf(sum.hi, kErrExp, wt * kErrArg); }
};

// Sum over the block; every thread gets it.
__device__ __forceinline__ Two block_add(Two a, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  a = warp_add(a);
  if (lane == 0) sh.part[warp] = a;
  __syncthreads();
  a = lane < warps ? sh.part[lane] : Two{0.f, 0.f};
  a = warp_add(a);
  __syncthreads();
  return a;
}
__device__ __forceinline__ float block_add(float a, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (lane == 0) sh.aux[warp] = a;
  __syncthreads();
  a = lane < warps ? sh.aux[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  __syncthreads();
  return a;
}

// The place of the last element to keep of those at or above `cut`: the
// `count` first of them (MASS false), or those before which less than `target`
// of weight stands (MASS).  `total`: how many elements there are.  In *loose the
// weight of the elements that may or may not belong (fp32 weights, whose sums
// are off by up to `err`).
//
// A histogram leaves an interval of the order with few enough elements to rank;
// the first one is over bins of equal width in z, later ones, where equal or
// nearly equal logits crowd a bin, over bins of equal width in the place.  The
// weights in it are whole multiples of a fixed step, so that sums do not depend
// on the order of the additions; the bins around the border are taken with a
// margin for that step.
template <bool MASS, bool TWO, typename T>
__device__ unsigned long long select(const Row<T>& r, Shared& sh, unsigned long long cut, int count, double target,
                                     float err, float* loose) {
  constexpr int kN = Vec<T>::kN;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
  // bins of the first histogram: 64 to a factor of two of the weight
  const float bin_scale = -64.f * r.scale.c_hi;
  auto bin_of = [&](float z) {
    return static_cast<int>(fminf((0.5f * z - r.scale.half_max) * bin_scale, static_cast<float>(kBins - 1)));
  };
  unsigned long long lo = 0, hi = ~0ull;  // the interval
  int shift = -1;                     // its bins' width; -1: the first histogram
  int n = r.V;                        // elements that the histogram counts, at most
  int before_n = 0;                   // elements ahead of the interval
  while (true) {
    const int digits = 31 - min(31, 32 - __clz(n));  // n elements of at most 2^digits
    const float one = static_cast<float>(1u << digits);
    // the heaviest weight in the interval
    const float top = shift < 0 ? 0.f : (0.5f * z_of(static_cast<uint32_t>(hi >> 32)) - r.scale.half_max) * r.scale.c_hi;
    for (int i = tid; i < kBins; i += nt) r.hist[i] = 0;
    __syncthreads();
    float ahead = 0.f;  // weight ahead of the interval
    each_of_part(r, [&](const float (&z)[kN], int id) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const unsigned long long p = place_of(key_of(z[i]), id + i);
        if (p < cut || id + i >= r.V) continue;
        int b;
        float t = 0.f;
        if (MASS) t = (0.5f * z[i] - r.scale.half_max) * r.scale.c_hi;
        if (shift < 0) {
          b = bin_of(z[i]);
          if (MASS) t += static_cast<float>(b) * 0.015625f;  // over the bin's first
        } else {
          if (p > hi) {
            if (MASS) ahead += ex2_approx(t);
            continue;
          }
          if (p < lo) continue;
          b = kBins - 1 - static_cast<int>((p - lo) >> shift);
          t -= top;
        }
        atomicAdd(&r.hist[b], MASS ? __float2uint_rn(fminf(ex2_approx(t), 1.f) * one) : 1u);
      }
    });
    if (MASS) ahead = block_add(ahead, sh);
    __syncthreads();
    // the bins that the border may be in
    const int per = kBins / nt;
    auto weight_of_bin = [&](int b) {
      const float w = static_cast<float>(r.hist[b]) / one;
      return shift < 0 ? ldexpf(exp2f(static_cast<float>(b & 63) * -0.015625f) * w, -(b >> 6)) : w * exp2f(top);
    };
    float mine = 0.f;
    int mine_n = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (MASS)
        mine += weight_of_bin(b);
      else
        mine_n += static_cast<int>(r.hist[b]);
    }
    float run = mine;
    int run_n = mine_n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float u = __shfl_up_sync(0xffffffffu, run, o);
      const int un = __shfl_up_sync(0xffffffffu, run_n, o);
      if (lane >= o) run += u, run_n += un;
    }
    if (lane == 31) {
      sh.aux[warp] = run;
      sh.num[warp] = run_n;
    }
    if (tid == 0) {
      sh.first = kBins - 1;
      sh.last = kBins - 1;
      sh.count = 0;
      sh.lo = 0xffffffffu;
      sh.hi = 0;
    }
    __syncthreads();
    float all = ahead;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) run += sh.aux[w], run_n += sh.num[w];
      all += sh.aux[w];
    }
    run += ahead - mine;
    run_n += before_n - mine_n;  // ahead of this thread's bins
    // a step of the histogram per element, and the roundings of the sums
    const float margin = MASS ? (shift < 0 ? all / one : static_cast<float>(n) / one * exp2f(top)) + 1e-5f * all + err : 0.f;
    const float want = static_cast<float>(target);
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (MASS) {
        const float next = run + weight_of_bin(b);
        if (next >= want - margin) atomicMin(&sh.first, b);
        if (next >= want + margin) atomicMin(&sh.last, b);
        run = next;
      } else {
        const int next = run_n + static_cast<int>(r.hist[b]);
        if (next >= count) {
          atomicMin(&sh.first, b);
          atomicMin(&sh.last, b);
        }
        run_n = next;
      }
    }
    __syncthreads();
    const int first = sh.first, last = sh.last;
    // the elements in them, and the weight ahead of them
    unsigned long long in_lo = 0, in_hi = 0;
    if (shift >= 0) {
      in_lo = lo + (static_cast<unsigned long long>(kBins - 1 - last) << shift);
      const unsigned long long off =
          (static_cast<unsigned long long>(kBins - 1 - first) << shift) + ((1ull << shift) - 1);
      in_hi = off >= hi - lo ? hi : lo + off;
    }
    Weights<TWO, T> above(r, sh.table);
    uint32_t k_lo = 0xffffffffu, k_hi = 0;
    int ahead_n = 0;
    each_of_part(r, [&](const float (&z)[kN], int id) {
      float zz[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t key = key_of(z[i]);
        const unsigned long long p = place_of(key, id + i);
        zz[i] = -INFINITY;
        if (p < cut || id + i >= r.V) continue;
        int where;  // 1 ahead, 0 in the interval, -1 behind
        if (shift < 0) {
          const int b = bin_of(z[i]);
          where = b < first ? 1 : b > last ? -1 : 0;
        } else {
          where = p > in_hi ? 1 : p < in_lo ? -1 : 0;
        }
        if (where > 0) {
          zz[i] = z[i];
          ++ahead_n;
        } else if (where == 0) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kList) r.list[at] = p;
          k_lo = min(k_lo, key);
          k_hi = max(k_hi, key);
        }
      }
      if (MASS) above.add_vec(zz, id, 1ull << 32);  // -inf weighs nothing
    });
    k_lo = __reduce_min_sync(0xffffffffu, k_lo);
    k_hi = __reduce_max_sync(0xffffffffu, k_hi);
    if (lane == 0) {
      atomicMin(&sh.lo, k_lo);
      atomicMax(&sh.hi, k_hi);
    }
    const Two ahead_w = MASS ? block_add(above.sum, sh) : Two{0.f, 0.f};
    ahead_n = __reduce_add_sync(0xffffffffu, ahead_n);
    if (lane == 0) sh.num[warp] = ahead_n;
    __syncthreads();
    ahead_n = 0;
    for (int w = 0; w < warps; ++w) ahead_n += sh.num[w];
    n = sh.count;
    if (n > kList) {
      const unsigned long long was = hi - lo;
      if (shift < 0) {
        lo = static_cast<unsigned long long>(sh.lo) << 32;
        hi = (static_cast<unsigned long long>(sh.hi) << 32) | 0xffffffffu;
      } else {
        lo = in_lo;
        hi = in_hi;
      }
      lo = max(lo, cut);
      if (lo >> 32 == hi >> 32) {  // one value: of its places the ids there are
        lo = max(lo, place_of(static_cast<uint32_t>(lo >> 32), r.V - 1));
        hi = min(hi, place_of(static_cast<uint32_t>(hi >> 32), 0));
      }
      before_n = ahead_n;
      if (MASS && hi - lo > was / 2) {
        // weights of very different sizes, too fine for the histogram's step: by halves
        const unsigned long long mid = lo + (hi - lo) / 2;
        Weights<TWO, T> w(r, sh.table);
        int more = 0;
        each_of_part(r, [&](const float (&z)[kN], int id) {
          w.add_vec(z, id, max(mid, cut));
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const unsigned long long p = place_of(key_of(z[i]), id + i);
            more += id + i < r.V && p >= mid && p <= hi;
          }
        });
        const double sum = value(block_add(w.sum, sh));
        more = __reduce_add_sync(0xffffffffu, more);
        if (lane == 0) sh.num[warp] = more;
        __syncthreads();
        more = 0;
        for (int x = 0; x < warps; ++x) more += sh.num[x];
        if (!TWO && fabs(sum - target) <= 2.0 * err) {  // left to the sums of two floats
          *loose = INFINITY;
          __syncthreads();
          return cut;
        }
        if (sum >= target) {
          lo = mid;
          n = more;
        } else {
          hi = mid - 1;
          n -= more;
          before_n += more;
        }
      }
      shift = max(0, 64 - __clzll(static_cast<long long>(hi - lo)) - 11);
      __syncthreads();
      continue;
    }
    // few enough: by rank
    for (int i = tid; i < n; i += nt) {
      const unsigned long long p = r.list[i];
      int rank = 0;
      for (int k = 0; k < n; ++k) rank += r.list[k] > p;
      r.sorted[rank] = p;
    }
    __syncthreads();
    if (!MASS) {
      const unsigned long long c = r.sorted[min(count - ahead_n, n) - 1];
      __syncthreads();
      return c;
    }
    if (warp == 0) {
      Two sum = ahead_w;  // of all before this round's
      int kept = 0;       // of the list
      float unsure = 0.f;
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        Two w{0.f, 0.f};
        if (i < n) {
          const float z = z_of(static_cast<uint32_t>(r.sorted[i] >> 32));
          float t;
          w = TWO ? weight2(r.scale, sh.table, z) : Two{weight1(r.scale, z, t), 0.f};
        }
        Two incl = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const Two u = shfl_up(incl, o);
          if (lane >= o) incl = add(incl, u);
        }
        incl = add(sum, incl);
        // weight before this element
        const double before = value(incl) - value(w);
        const bool in = i < n && before < target;
        kept += __popc(__ballot_sync(0xffffffffu, in));
        if (!TWO && i < n && fabs(before - target) <= 2.0 * err) unsure += w.hi;
        sum = {__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)};
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) unsure += __shfl_xor_sync(0xffffffffu, unsure, o);
      if (lane == 0) {
        // (with the margin the list's first is in; where nothing is ahead of it it is kept anyway)
        sh.cut = r.sorted[max(kept, 1) - 1];
        sh.loose = unsure;
      }
    }
    __syncthreads();
    *loose = sh.loose;
    const unsigned long long c = sh.cut;
    __syncthreads();
    return c;
  }
}

// Draws the row's token from the elements at or above `cut`, of those the first
// that top_p leaves, and at or above cut_min.  False where fp32 sums do not
// decide it.
template <bool TWO, typename T>
__device__ bool draw(const Row<T>& r, Shared& sh, unsigned long long cut, unsigned long long cut_min, float top_p,
                     float u, int& token, float& logprob) {
  constexpr int kN = Vec<T>::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  float loose = 0.f;
  if (top_p < 1.f) {
    Weights<TWO, T> w(r, sh.table);
    each_of_part(r, [&](const float (&z)[kN], int id) { w.add_vec(z, id, cut); });
    const Two all = block_add(w.sum, sh);
    const float err = TWO ? 0.f : block_add(w.error(), sh);
    const unsigned long long c =
        select<true, TWO>(r, sh, cut, 0, static_cast<double>(top_p) * value(all), err, &loose);
    cut = max(cut, c);
  }
  cut = max(cut, cut_min);
  // the sums of the warps' parts
  Weights<TWO, T> w(r, sh.table);
  each_of_part(r, [&](const float (&z)[kN], int id) { w.add_vec(z, id, cut); });
  const float err = (TWO ? 0.f : block_add(w.error(), sh)) + loose;
  Two part = warp_add(norm(w.sum.hi, w.sum.lo));
  if (lane == 0) sh.part[warp] = part;
  __syncthreads();
  part = lane < warps ? sh.part[lane] : Two{0.f, 0.f};
  Two incl = part;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two up = shfl_up(incl, o);
    if (lane >= o) incl = add(incl, up);
  }
  const Two all{__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)};
  const double target = static_cast<double>(u) * value(all);
  __syncthreads();
  // the first part whose end passes the target (the last that has weight, where rounding leaves none)
  auto first_past = [&](const Two& end, bool has) {
    const unsigned past = __ballot_sync(0xffffffffu, has && value(end) > target);
    if (past) return __ffs(static_cast<int>(past)) - 1;
    const unsigned any = __ballot_sync(0xffffffffu, has);
    return any ? 31 - __clz(static_cast<int>(any)) : 0;
  };
  const int w0 = first_past(incl, part.hi > 0.f);
  Two before{__shfl_sync(0xffffffffu, incl.hi, (w0 + 31) & 31), __shfl_sync(0xffffffffu, incl.lo, (w0 + 31) & 31)};
  if (w0 == 0) before = {0.f, 0.f};
  // that part of the row, cut among the warps in the same way
  const int from = w0 * r.per_warp, to = min(from + r.per_warp, r.vecs);
  const int step = ((to - from + warps - 1) / warps + 31) / 32 * 32;
  const int a = min(from + warp * step, to), b = min(a + step, to);
  Weights<TWO, T> w1(r, sh.table);
  each(r, a, b, [&](const float (&z)[kN], int id) { w1.add_vec(z, id, cut); });
  part = warp_add(norm(w1.sum.hi, w1.sum.lo));
  if (lane == 0) sh.part[warp] = part;
  __syncthreads();
  part = lane < warps ? sh.part[lane] : Two{0.f, 0.f};
  incl = part;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two up = shfl_up(incl, o);
    if (lane >= o) incl = add(incl, up);
  }
  incl = add(before, incl);
  const int w2 = first_past(incl, part.hi > 0.f);
  if (w2 > 0)
    before = {__shfl_sync(0xffffffffu, incl.hi, w2 - 1), __shfl_sync(0xffffffffu, incl.lo, w2 - 1)};
  if (warp == 0) {  // and that one, vector by vector
    const int v0 = from + w2 * step, v1 = min(v0 + step, to);
    int found = -1;
    float margin = 0.f, z_found = 0.f;
    for (int v = v0; v < v1; v += 32) {
      Weights<TWO, T> one(r, sh.table);
      each(r, v, min(v + 32, v1), [&](const float (&z)[kN], int id) { one.add_vec(z, id, cut); });
      const Two mine = norm(one.sum.hi, one.sum.lo);
      incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Two up = shfl_up(incl, o);
        if (lane >= o) incl = add(incl, up);
      }
      incl = add(before, incl);
      const unsigned has = __ballot_sync(0xffffffffu, mine.hi > 0.f);
      const unsigned past = __ballot_sync(0xffffffffu, mine.hi > 0.f && value(incl) > target);
      // (the last one that has weight, as long as no later one passes the target)
      const int l = past ? __ffs(static_cast<int>(past)) - 1 : has ? 31 - __clz(static_cast<int>(has)) : -1;
      if (l >= 0) {
        Two run{__shfl_sync(0xffffffffu, incl.hi, (l + 31) & 31), __shfl_sync(0xffffffffu, incl.lo, (l + 31) & 31)};
        if (l == 0) run = before;
        const int vec = v + l;
        float z[kN];
        Vec<T>::unpack(r.v[vec], z);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int id = vec * kN + i;
          if (id >= r.V || place_of(key_of(z[i]), id) < cut) continue;
          float t;
          const Two x = TWO ? weight2(r.scale, sh.table, z[i]) : Two{weight1(r.scale, z[i], t), 0.f};
          if (!(x.hi > 0.f)) continue;
          const double start = value(run);
          run = add(run, x);
          if (found < 0 || start <= target) {
            found = id;
            z_found = z[i];
            // how far the random number is from the ends of this token's share (nothing is before the first)
            margin = static_cast<float>(value(run) - target);
            if (start > 0.0 || loose > 0.f) margin = fminf(margin, static_cast<float>(target - start));
          }
        }
      }
      before = {__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)};
      if (past) break;
    }
    if (lane == 0) {
      sh.found = found;
      const double t = (0.5 * z_found - static_cast<double>(r.scale.half_max)) *
                       (static_cast<double>(r.scale.c_hi) + r.scale.c_lo);
      sh.before = 0.693147180559945f * (static_cast<float>(t) - log2f(all.hi));
      sh.loose = margin;
    }
  }
  __syncthreads();
  token = sh.found;
  logprob = sh.before;
  const float margin = sh.loose;
  __syncthreads();
  return TWO || (margin > 2.f * err && loose <= 4e-6f * all.hi);
}

template <typename T, int NT, bool IN_SMEM>
__global__ void __launch_bounds__(NT, NT == 1024 ? 1 : NT == 512 ? 2 : 8) sample_rows(const SampleArgs a) {
  constexpr int kN = Vec<T>::kN;
  extern __shared__ __align__(16) uint8_t s_raw[];
  __shared__ Shared sh;
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long m = blockIdx.x;
  Row<T> r;
  r.V = a.V;
  r.vecs = (a.V + kN - 1) / kN;
  r.per_warp = ((r.vecs + NT / 32 - 1) / (NT / 32) + 31) / 32 * 32;
  r.hist = reinterpret_cast<uint32_t*>(s_raw);
  r.sorted = reinterpret_cast<unsigned long long*>(s_raw);
  r.list = reinterpret_cast<unsigned long long*>(s_raw + kBins * 4);
  uint4* kept = reinterpret_cast<uint4*>(s_raw + kBins * 4 + kList * 8);
  const uint4* global = reinterpret_cast<const uint4*>(static_cast<const T*>(a.logits) + m * a.ld);
  r.v = IN_SMEM ? kept : global;
  for (int i = tid; i < 65; i += NT) sh.table[i] = kExp2[i];
  if (tid == 0) s_bad = 0;
  griddep_wait();
  griddep_launch_dependents();
  // the row, its maximum, and whether it has a NaN or +inf
  float top = -INFINITY;
  bool bad = false;
  {
    const int from = min(warp * r.per_warp, r.vecs), to = min(from + r.per_warp, r.vecs);
#pragma unroll 4
    for (int v = from + lane; v < to; v += 32) {
      const uint4 u = global[v];
      if (IN_SMEM) kept[v] = u;
      float z[kN];
      Vec<T>::unpack(u, z);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        if (v * kN + i >= a.V) z[i] = -INFINITY;
        top = fmaxf(top, z[i]);
        bad |= !(z[i] < INFINITY);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  __syncthreads();
  if (lane == 0) sh.aux[warp] = top;
  if (bad) s_bad = 1;
  __syncthreads();
  top = lane < NT / 32 ? sh.aux[lane] : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  top += 0.f;
  bad = s_bad != 0 || top == -INFINITY;
  const float temperature = a.temperature ? a.temperature[m] : 1.f, top_p = a.top_p ? a.top_p[m] : 1.f,
              min_p = a.min_p ? a.min_p[m] : 0.f, u = a.uniform[m];
  const int top_k = a.top_k ? a.top_k[m] : 0;
  const bool wrong = !(temperature >= 0.f && temperature < INFINITY) || top_k < 0 || !(top_p >= 0.f) ||
                     !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f);
  int token = -1;
  float logprob = __int_as_float(0x7fffffff);
  if (wrong) {
    if (tid == 0) record_error(a.err, kErrRange, kSiteSampleRow);
  } else if (!bad && (temperature == 0.f || top_k == 1 || top_p == 0.f)) {
    // the first of the order alone
    __syncthreads();
    int first = a.V;
    each_of_part(r, [&](const float (&z)[kN], int id) {
#pragma unroll
      for (int i = kN - 1; i >= 0; --i)
        if (z[i] == top) first = min(first, id + i);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.num[warp] = first;
    __syncthreads();
    for (int w = 0; w < NT / 32; ++w) first = min(first, sh.num[w]);
    token = first;
    logprob = 0.f;
  } else if (!bad) {
    // 2 log2(e) / temperature
    const double c = 2.8853900817779268 / fmin(fmax(static_cast<double>(temperature), 0x1p-100), 0x1p100);
    r.scale.half_max = 0.5f * top;
    r.scale.c_hi = static_cast<float>(c);
    r.scale.c_lo = static_cast<float>(c - r.scale.c_hi);
    unsigned long long cut = 0, cut_min = 0;
    if (min_p > 0.f) {
      // the least z with z - max >= temperature log(min_p)
      const double least = static_cast<double>(temperature) * log(static_cast<double>(min_p));
      float z = static_cast<float>(top + least);
      if (!(z >= -3.402823466e38f)) z = -3.402823466e38f;
      auto in = [&](float x) { return static_cast<double>(x) - top >= least; };
      // (one step at most, unless z is so small beside the maximum that the difference does not show it)
      for (int i = 0; i < 4 && z > -3.402823466e38f && in(nextafterf(z, -INFINITY)); ++i) z = nextafterf(z, -INFINITY);
      for (int i = 0; i < 4 && !in(z); ++i) z = nextafterf(z, INFINITY);
      cut_min = static_cast<unsigned long long>(key_of(z)) << 32;
    }
    __syncthreads();
    if (top_k > 0 && top_k < a.V) cut = select<false, false>(r, sh, 0ull, top_k, 0.0, 0.f, nullptr);
    if (!draw<false>(r, sh, cut, cut_min, top_p, u, token, logprob))
      draw<true>(r, sh, cut, cut_min, top_p, u, token, logprob);
  }
  if (tid == 0) {
    a.tokens[m] = token;
    if (a.logprob) a.logprob[m] = logprob;
  }
}

// Threads per row: many rows that are short keep the SM busy with several CTAs,
// a row that fills its shared memory with one.
template <typename T, int NT, bool IN_SMEM>
cudaError_t launch_nt(const SampleArgs& a, int64_t M, size_t smem, cudaStream_t s) {
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(sample_rows<T, NT, IN_SMEM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         227 * 1024 - 2048);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  return launch_pdl(sample_rows<T, NT, IN_SMEM>, static_cast<unsigned>(M), NT, smem, s, 0, a);
}
template <typename T>
cudaError_t launch_type(const SampleArgs& a, int64_t M, cudaStream_t s) {
  const size_t row = (static_cast<size_t>(a.V) * sizeof(T) + 15) / 16 * 16, fixed = kBins * 4 + kList * 8;
  if (row <= 16 * 1024) return launch_nt<T, 128, true>(a, M, fixed + row, s);
  if (row + fixed <= 112 * 1024 - 2048) return launch_nt<T, 512, true>(a, M, fixed + row, s);
  if (row + fixed <= 227 * 1024 - 2048) return launch_nt<T, 1024, true>(a, M, fixed + row, s);
  return launch_nt<T, 1024, false>(a, M, fixed, s);
}

}  // namespace

cudaError_t launch_sample_tokens(const void* logits, int64_t ld, gpt2_dtype logits_t, int64_t M, int V,
                                 const float* temperature, const int32_t* top_k, const float* top_p,
                                 const float* min_p, const float* uniform, int32_t* tokens, float* logprob,
                                 cudaStream_t s) {
  const SampleArgs a{logits, ld, V, temperature, top_k, top_p, min_p, uniform, tokens, logprob, device_error_word()};
  if (logits_t == GPT2_F32) return launch_type<float>(a, M, s);
  if (logits_t == GPT2_F16) return launch_type<__half>(a, M, s);
  return launch_type<__nv_bfloat16>(a, M, s);
}

}  // namespace gpt2
